"""The oracle's layer norm, gated norm and gated linear recurrence against torch's
automatic differentiation of the same formulas, written apart, in 64 bits (CPU)."""
import pytest

torch = pytest.importorskip("torch")

from oracle import layer as L

F64 = torch.float64


def rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def leaf(*shape, seed):
    return rnd(*shape, seed=seed).requires_grad_()


def near(a, b):
    assert torch.allclose(a, b, rtol=1e-9, atol=1e-11)


def test_layer_norm():
    x, w, b, dy, dres = leaf(5, 12, seed=1), leaf(12, seed=2), leaf(12, seed=3), rnd(5, 12, seed=4), rnd(5, 12, seed=5)
    y = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-3) * w + b
    ((y * dy).sum() + (x * dres).sum()).backward()
    got, s, _ = L.layer_norm(x, w, b, None, 1e-3)
    near(got, y.detach())
    ds, dw, db = L.layer_norm_grad(dy, s, w, dres, 1e-3)
    near(ds, x.grad)
    near(dw, w.grad)
    near(db, b.grad)


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gate_norm(first, center, act):
    x, z, w, b, dy = leaf(4, 3, 8, seed=1), leaf(4, 3, 8, seed=2), leaf(3, 8, seed=3), leaf(3, 8, seed=4), rnd(4, 3, 8, seed=5)
    a = torch.nn.functional.silu(z) if act == "silu" else torch.sigmoid(z)
    v = x * a if first else x
    if center:
        n = torch.nn.functional.layer_norm(v, (8,), eps=1e-3) * w + b
    else:
        n = v * (v.square().mean(-1, keepdim=True) + 1e-3).rsqrt() * w
    y = n if first else n * a
    (y * dy).sum().backward()
    out = L.gate_norm(x, z, w, b if center else None, 1e-3, act, first, center, dy)
    near(out["y"], y.detach())
    for name, t in (("dx", x), ("dz", z), ("dw", w)) + ((("db", b),) if center else ()):
        near(out[name], t.grad)
    for name in ("y", "dx", "dz", "dw", "db"):          # sizes are no less than what they are sizes of
        assert (out[name].abs() <= out[name + "size"] * (1 + 1e-12)).all(), name


@pytest.mark.parametrize("form", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("scale", [None, "complement", "norm"])
def test_glr(form, scale):
    lens, T, D = [3, 0, 7, 1], 11, 4
    x, g, h0, dy, dhT = leaf(T, D, seed=1), leaf(T, D, seed=2), leaf(4, D, seed=3), rnd(T, D, seed=4), rnd(4, D, seed=5)
    bias = leaf(D, seed=6)
    rate = (0.1 + rnd(D, seed=7).abs()).requires_grad_() if form == "rate" else None
    v = g + bias if form != "log" else -(g + bias).abs()
    a = torch.exp(v) if form == "log" else torch.sigmoid(v) if form == "sigmoid" else torch.exp(-rate * torch.sigmoid(v))
    c = 1.0 if scale is None else 1 - a if scale == "complement" else torch.sqrt(1 - a * a)
    h, ys, ends, at = None, [], [], 0
    for n, m in enumerate(lens):
        h = h0[n]
        for t in range(at, at + m):
            h = a[t] * h + (c * x)[t]
            ys.append(h)
        ends.append(h)
        at += m
    y, hT = torch.stack(ys), torch.stack(ends)
    ((y * dy).sum() + (hT * dhT).sum()).backward()
    raw = v.detach() - (0 if form == "log" else bias.detach())
    out = L.glr(x, raw, None if form == "log" else bias, rate, h0, lens, form, scale, dy, dhT)
    near(out["y"], y.detach())
    near(out["hT"], hT.detach())
    near(out["dx"], x.grad)
    near(out["dh0"], h0.grad)
    sign = -torch.sign((g + bias).detach()) if form == "log" else 1.0
    near(out["dgate"] * sign, g.grad)
    near((out["dgate"] * sign).sum(0), bias.grad)
    if form == "rate":
        near(out["drate"], rate.grad)
    for k in ("y", "hT", "dx", "dgate", "dh0", "dbias", "drate"):
        assert (out[k + "_err"] >= 0).all() and out[k + "_err"].shape == out[k].shape
