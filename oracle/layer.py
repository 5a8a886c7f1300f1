"""The layer operators from their definitions, token by token in 64 bits (torch
on the CPU): the root-mean-square norm, layer norm, the gated norm, the short
causal convolution, the selective state space scan and the gated linear
recurrence, with their gradients.

Every scan and convolution takes packed rows and ``lens``, the sequences'
lengths: x [T, ...] holds the sequences one behind the other, a state per
sequence.  ``absolute`` replaces every factor by its size, so that a result is
the sum of its terms' sizes: what rounding errors are measured against.
"""
import torch

F64 = torch.float64


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def norm(x, weight, residual, eps, keep=None):
    """(y, s): s is rounded to ``keep`` (the residual's type) before the norm."""
    s = f64(x)
    if residual is not None:
        s = (x.cpu().float() + residual.cpu().float()).to(keep).to(F64)
    r = (s.square().mean(-1, keepdim=True) + eps).rsqrt()
    return s * r * f64(weight), s


def norm_grad(dy, s, weight, dres, eps):
    """(ds, dw) for s as kept."""
    dy, s, w = f64(dy), f64(s), f64(weight)
    r = (s.square().mean(-1, keepdim=True) + eps).rsqrt()
    u = dy * w
    ds = r * (u - s * r * r * (u * s).mean(-1, keepdim=True))
    if dres is not None:
        ds = ds + f64(dres)
    return ds, (dy * s * r).reshape(-1, s.shape[-1]).sum(0)


def _lines(x, state, lens, W):
    """Per sequence: its state's rows and its own."""
    at = 0
    for n, k in enumerate(lens):
        before = torch.zeros(W - 1, x.shape[1], dtype=F64) if state is None else state[n]
        yield n, at, k, torch.cat([before, x[at:at + k]])
        at += k


def conv(x, weight, bias, state, lens, silu, absolute=False):
    """(y [T, D], final states [n, W-1, D])."""
    x, w, b, state = f64(x), f64(weight), f64(bias), f64(state)
    if absolute:
        x, w, b, state = x.abs(), w.abs(), None if b is None else b.abs(), None if state is None else state.abs()
    W = w.shape[1]
    y, last = torch.zeros_like(x), []
    for n, at, k, line in _lines(x, state, lens, W):
        v = sum(w[:, j] * line[j:j + k] for j in range(W)) + (0 if b is None else b)
        y[at:at + k] = v * torch.sigmoid(v) if silu and not absolute else v
        last.append(line[k:])
    return y, torch.stack(last)


def conv_grad(dy, x, weight, bias, state, lens, silu, dfinal, absolute=False):
    """(dx, dw, db, dstate)."""
    dy, x, w, b, state, dfinal = (f64(t) for t in (dy, x, weight, bias, state, dfinal))
    if absolute:
        dy, x, w, b, state, dfinal = (None if t is None else t.abs() for t in (dy, x, w, b, state, dfinal))
    W = w.shape[1]
    dx, dw, db, ds = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w[:, 0]), []
    for n, at, k, line in _lines(x, state, lens, W):
        v = sum(w[:, j] * line[j:j + k] for j in range(W)) + (0 if b is None else b)
        dv = dy[at:at + k]
        if silu and not absolute:
            g = torch.sigmoid(v)
            dv = dv * (g + v * g * (1 - g))
        elif silu:
            dv = dv * 1.1                       # |silu'| stays below that
        dline = torch.zeros_like(line)
        for j in range(W):
            dline[j:j + k] += w[:, j] * dv
            dw[:, j] += (dv * line[j:j + k]).sum(0)
        db += dv.sum(0)
        if dfinal is not None:
            dline[k:] += dfinal[n]
        ds.append(dline[:W - 1])
        dx[at:at + k] = dline[W - 1:]
    return dx, dw, db, torch.stack(ds)


def step_sizes(dt, dt_bias, softplus):
    raw = f64(dt) + (0 if dt_bias is None else f64(dt_bias))
    return torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw, raw


def ssm(x, dt, A, B, C, D, h0, lens, absolute=False, keep=None):
    """(y [T, H, P], final states [n, H, N, P]); dt as used (step_sizes).  With
    ``keep`` a list, every state is appended to it, the first one included."""
    x, dt, A, B, C, D, h0 = (f64(t) for t in (x, dt, A, B, C, D, h0))
    if absolute:
        x, B, C, D, h0 = (None if t is None else t.abs() for t in (x, B, C, D, h0))
    T, H, P = x.shape
    G, N = B.shape[1:]
    Bh, Ch = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    y, last, at = torch.zeros_like(x), [], 0
    for n, k in enumerate(lens):
        h = torch.zeros(H, N, P, dtype=F64) if h0 is None else h0[n]
        states = [h]
        for t in range(at, at + k):
            h = torch.exp(dt[t] * A)[:, None, None] * h + Bh[t][:, :, None] * (dt[t][:, None] * x[t])[:, None, :]
            y[t] = torch.matmul(Ch[t][:, None, :], h)[:, 0] + (0 if D is None else D[:, None] * x[t])
            states.append(h)
        if keep is not None:
            keep.append(states)
        last.append(h)
        at += k
    return y, torch.stack(last)


def ssm_grad(dy, x, dt, A, B, C, D, h0, lens, dhT, absolute=False):
    """dict of dx, ddt (of dt as used), dA, dB, dC, dD, dh0; with ``absolute``
    every sum of its terms' sizes, and "pairs": per token and head, the size of
    all pairs that meet the token."""
    keep = []
    ssm(x, dt, A, B, C, D, h0, lens, absolute, keep)
    dy, x, dt, A, B, C, D, dhT = (f64(t) for t in (dy, x, dt, A, B, C, D, dhT))
    if absolute:
        dy, x, B, C, D, dhT = (None if t is None else t.abs() for t in (dy, x, B, C, D, dhT))
    T, H, P = x.shape
    G, N = B.shape[1:]
    Bh, Ch = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    fold = lambda v: v.unflatten(0, (G, H // G)).sum(1)  # noqa: E731
    out = dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(dt), dA=torch.zeros_like(A), dB=torch.zeros_like(B),
               dC=torch.zeros_like(C), dD=(dy * x).sum((0, 2)), dh0=[], pairs=torch.zeros_like(dt))
    at = 0
    for n, k in enumerate(lens):
        dh = torch.zeros(H, N, P, dtype=F64) if dhT is None else dhT[n]
        for t in reversed(range(at, at + k)):
            h, prev = keep[n][t - at + 1], keep[n][t - at]
            dC = torch.matmul(h, dy[t][:, :, None])[..., 0]
            out["dC"][t] = fold(dC)
            dh = dh + Ch[t][:, :, None] * dy[t][:, None, :]
            du = torch.matmul(Bh[t][:, None, :], dh)[:, 0]
            out["dx"][t] = dt[t][:, None] * du + (0 if D is None else D[:, None] * dy[t])
            out["dB"][t] = fold(torch.matmul(dh, (dt[t][:, None] * x[t])[:, :, None])[..., 0])
            a = torch.exp(dt[t] * A)
            dg = (dh * prev).sum((1, 2)) * a
            c = (du * x[t]).sum(1)
            out["ddt"][t] = c + dg * (A.abs() if absolute else A)
            out["dA"] += dg * dt[t]
            out["pairs"][t] = dt[t] * c + (dC * Ch[t]).sum(1) + dg
            dh = dh * a[:, None, None]
        out["dh0"].append(dh)
        at += k
    out["dh0"] = torch.stack(out["dh0"])
    return out


def layer_norm(x, weight, bias, residual, eps, keep=None):
    """(y, s, h): s is rounded to ``keep`` (the residual's type) before the norm; h is
    s less its mean, over its deviation."""
    s = f64(x)
    if residual is not None:
        s = (x.cpu().float() + residual.cpu().float()).to(keep).to(F64)
    v = s - s.mean(-1, keepdim=True)
    h = v * (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    return h * f64(weight) + (0 if bias is None else f64(bias)), s, h


def layer_norm_grad(dy, s, weight, dres, eps):
    """(ds, dw, db) for s as kept."""
    dy, s, w = f64(dy), f64(s), f64(weight)
    v = s - s.mean(-1, keepdim=True)
    r = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    h, u = v * r, dy * w
    ds = r * (u - u.mean(-1, keepdim=True) - h * (u * h).mean(-1, keepdim=True))
    if dres is not None:
        ds = ds + f64(dres)
    D = s.shape[-1]
    return ds, (dy * h).reshape(-1, D).sum(0), dy.reshape(-1, D).sum(0)


def gate_norm(x, z, weight, bias, eps, act, first, center, dy=None):
    """dict of y, its terms' sizes ysize, and with dy (like x) of dx, dz, dw, db and their
    sizes, for rows x [T, H, D]; dw and db are [H, D], one for each head."""
    x, z, w, b = f64(x), f64(z), f64(weight), 0.0 if bias is None else f64(bias)
    g, o = torch.sigmoid(z), torch.sigmoid(-z)
    a, da = (z * g, g + z * g * o) if act == "silu" else (g, g * o)
    dasize = g + z.abs() * g * o if act == "silu" else g * o
    one = 1.0 if center else 0.0          # a mean's error is of the size of a deviation
    v = x * a if first else x
    if center:
        v = v - v.mean(-1, keepdim=True)
    r = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = v * r
    n, nsize = h * w + b, (h.abs() + one) * w.abs() + (b.abs() if center and bias is not None else 0)
    out = dict(y=n if first else n * a, ysize=nsize if first else nsize * a.abs())
    if dy is None:
        return out
    dy = f64(dy)
    dn = dy if first else dy * a
    u = dn * w
    dv = u - h * (u * h).mean(-1, keepdim=True)
    size = u.abs() + (h.abs() + one) * (u.abs() * (h.abs() + one)).mean(-1, keepdim=True)
    if center:
        dv, size = dv - u.mean(-1, keepdim=True), size + u.abs().mean(-1, keepdim=True)
    dv, size = r * dv, r * size
    out.update(dx=dv * a if first else dv, dxsize=size * a.abs() if first else size,
               dz=dv * x * da if first else dy * n * da, dzsize=size * x.abs() * dasize if first else dy.abs() * nsize * dasize,
               dw=(dn * h).sum(0), dwsize=(dn.abs() * (h.abs() + one)).sum(0), db=dn.sum(0), dbsize=dn.abs().sum(0))
    return out


def glr_gates(gate, bias, rate, form, scale):
    """a, c = 1 - a, the input's factor k and its derivative by log a, d(log a)/d(gate), sigmoid."""
    v = f64(gate) + (0 if bias is None else f64(bias))
    if form == "log":
        a, c, slope, g = torch.exp(v), -torch.expm1(v), torch.ones_like(v), torch.zeros_like(v)
    else:
        g, o = torch.sigmoid(v), torch.sigmoid(-v)
        la = torch.nn.functional.logsigmoid(v) if form == "sigmoid" else -f64(rate) * g
        a, c = (g, o) if form == "sigmoid" else (torch.exp(la), -torch.expm1(la))
        slope = o if form == "sigmoid" else la * o
    if scale is None:
        return a, c, torch.ones_like(a), torch.zeros_like(a), slope, g
    if scale == "complement":
        return a, c, c, -a, slope, g
    k = torch.sqrt(c * (1 + a))
    return a, c, k, torch.where(k > 0, -a * a / k, torch.zeros_like(k)), slope, g


UNIT = 2.0 ** -24


def glr(x, gate, bias, rate, h0, lens, form, scale, dy=None, dhT=None):
    """The recurrence over packed rows [T, D] of sequences of ``lens`` tokens: dict of
    y, hT, and with dy of dx, dgate, dbias, drate, dh0.  For each name, name + "_err" is what
    fp32 may be off: every token's state may be rounded by 2 units of its terms' sizes S, and
    be off by 16 units of what the token takes from it (c S) and adds to it (|u|), the
    errors of the gate's functions and of the moves that lack c to 1; products take 16 units more."""
    x, h0, dy, dhT = f64(x), f64(h0), f64(dy), f64(dhT)
    a, c, k, dk, slope, g = glr_gates(gate, bias, rate, form, scale)
    T, D = x.shape
    u = k * x
    y, ey, sizes = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    prev, eprev, sprev = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    hT, ehT, at = [], [], 0
    zero = torch.zeros(D, dtype=F64)
    for n, m in enumerate(lens):
        h = zero if h0 is None else h0[n]
        s, e = h.abs(), zero
        for t in range(at, at + m):
            prev[t], eprev[t], sprev[t] = h, e, s
            e = a[t] * e + UNIT * 16 * (c[t].abs() * s + u[t].abs())
            h, s = a[t] * h + u[t], a[t] * s + u[t].abs()
            e = e + UNIT * 2 * s
            y[t], ey[t], sizes[t] = h, e, s
        hT.append(h)
        ehT.append(e)
        at += m
    out = dict(y=y, y_err=2 * ey, hT=torch.stack(hT), hT_err=2 * torch.stack(ehT))
    if dy is None:
        return out
    dx, da, ex, eda, dasize = (torch.zeros_like(x) for _ in range(5))
    dh0, edh0 = [], []
    at = T if sum(lens) == T else sum(lens)
    for n in reversed(range(len(lens))):
        d = zero if dhT is None else dhT[n]
        s, e = d.abs(), zero
        for t in reversed(range(at - lens[n], at)):
            d, s = d + dy[t], s + dy[t].abs()
            e = e + UNIT * 2 * s
            dx[t], ex[t] = d * k[t], k[t].abs() * (e + UNIT * 16 * s)
            size = a[t] * s * sprev[t] + s * (x[t] * dk[t]).abs()
            da[t], dasize[t] = a[t] * d * prev[t] + d * x[t] * dk[t], size
            eda[t] = a[t] * (e * sprev[t] + s * eprev[t]) + e * (x[t] * dk[t]).abs() + 32 * UNIT * size
            e = a[t] * e + UNIT * 16 * c[t].abs() * s
            d, s = a[t] * d, a[t] * s
            e = e + UNIT * s
        dh0.insert(0, d)
        edh0.insert(0, e)
        at -= lens[n]
    out.update(dx=dx, dx_err=2 * ex, dgate=da * slope, dgate_err=2 * slope.abs() * (eda + 16 * UNIT * dasize),
               dh0=torch.stack(dh0), dh0_err=2 * torch.stack(edh0))
    # sums of a tile's runs (8), groups and waves (10), then of the tiles in 64 lines
    many = UNIT * (32 + 64 + len(x) / 64)
    out.update(dbias=out["dgate"].sum(0), dbias_err=out["dgate_err"].sum(0) + many * (dasize * slope.abs()).sum(0),
               drate=-(da * g).sum(0), drate_err=2 * (eda * g).sum(0) + (many + 16 * UNIT) * (dasize * g).sum(0))
    return out
