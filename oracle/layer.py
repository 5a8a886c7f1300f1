"""The layer operators from their definitions, token by token in 64 bits (torch
on the CPU): the root-mean-square norm, the short causal convolution and the
selective state space scan, with their gradients.

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
