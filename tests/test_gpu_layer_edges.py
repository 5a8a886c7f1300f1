"""Values at the edges of what the layer operators take: NaN in 8-bit rows, decays next to 1,
gates that their bias cancels; against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ARITH = 2.0 ** -18          # of a row's terms, as in test_gpu_layer_norms.py


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def close(got, ref, tol, what):
    d = (got.detach().cpu().double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e over its tolerance" % (what, int(bad.sum()), bad.numel(),
                                                                               float((d - tol).max()))


@pytest.mark.parametrize("D", [129, 130, 132, 401])
@pytest.mark.parametrize("first,n", [(0, 64), (64, 64), (3, 1), (0, 128)])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("group", [0, 128])
def test_a_nan_does_not_enter_the_scale(D, first, n, centered, group):
    """NaN weights make n columns NaN: they stay NaN, and the others have the scale that they
    have by themselves."""
    x, w = rnd(3, D, seed=1), rnd(D, seed=2, scale=0.2) + 1
    bad = w.clone()
    bad[first:first + n] = float("nan")
    f = gdn.layer_norm_forward if centered else gdn.norm_forward
    q, _, scale = f(x, bad, out_dtype=FP8, group=group, eps=1e-5)
    v = x.cpu().double()
    v = v - v.mean(-1, keepdim=True) if centered else v
    h = v * (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    ref = h * w.cpu().double()
    ref[:, first:first + n] = 0
    size = (h.abs() + 1) * w.cpu().double().abs() * ARITH
    size[:, first:first + n] = 0
    g = group or D
    cols = [slice(k, min(k + g, D)) for k in range(0, D, g)]
    amax, slack = (torch.stack([t[:, c].abs().amax(1) for c in cols], 1) / 448 for t in (ref, size))
    want = amax.clamp(min=2.0 ** -126)
    close(scale, want, want * ARITH + slack, "scale")
    got = q.float().cpu().double()
    assert got[:, first:first + n].isnan().all()
    got[:, first:first + n] = 0
    full = scale.cpu().double().repeat_interleave(g, 1)[:, :D]
    u = ref / full
    # half a step of e4m3, whose subnormals are 2^-9 apart
    close(got, u, u.abs() * (2.0 ** -4 + ARITH) + 2.0 ** -10 + size / full, "q")


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------

HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = 2.0 ** -120


def glr_close(got, ref, names):
    for name, v in zip(names, got):
        if v is not None:
            r = ref[name]
            close(v.reshape(r.shape), r, ref[name + "_err"] + r.abs() * HALF[v.dtype] + TINY, name)


@pytest.mark.parametrize("dt,gt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("D", [64, 65])
@pytest.mark.parametrize("scale", [None, "complement", "norm"])
def test_decays_next_to_one(dt, gt, D, scale):
    """Log decays down to the least denormal number (log sigmoid of 88 and more is one): 1 - a is
    the gate itself, sqrt(1 - a^2) = sqrt(-2 gate), its derivative -1 / sqrt(-2 gate); from
    1 - a^2 < 2^-126 on both are 0, as for a gate of 0.  Each tolerance is the oracle's, relative
    errors of fp32."""
    T = 40
    sizes = [0.0, 1e-36, 1e-37, 2.0 ** -126, 2.0 ** -127, 1e-38, 1e-39, 8e-40, 2.0 ** -133, 0.0]
    gate = -torch.tensor([[sizes[(t + c) % 10] if t % 13 else 0.1 for c in range(D)] for t in range(T)]).to(gt).to(DEV)[None]
    if gt == F32:
        gate[0, 7] = -2.0 ** -149
    taken = gate if scale != "norm" else torch.where(gate > -2.0 ** -127, torch.zeros_like(gate), gate)
    x, dy = rnd(1, T, D, seed=1, dtype=dt), rnd(1, T, D, seed=2, dtype=dt)
    for h0 in (rnd(1, D, seed=3), None):
        dhT = None if h0 is None else rnd(1, D, seed=4)
        y, hT = gdn.glr_forward(x, gate, h0, scale=scale)
        grads = gdn.glr_backward(dy, x, gate, h0, dhT, scale=scale)
        ref = L.glr(x[0], taken[0], None, None, h0, [T], "log", scale, dy[0], dhT)
        glr_close((y, hT, *grads), ref, ("y", "hT", "dx", "dgate", "dbias", "drate", "dh0"))
    # from nothing: the inputs alone, whose factors are as small as 2^-63
    first = gate[0, 1:11].contiguous()
    state, one = torch.zeros(10, D, device=DEV), x[0, 1:11]
    y = gdn.glr_step(one, first, state, scale=scale)
    ref = L.glr(one, taken[0, 1:11], None, None, None, [1] * 10, "log", scale)
    glr_close((y, state), ref, ("y", "hT"))


def test_rates_of_far_gates():
    """log a = -rate sigmoid(v) with v as far as -82, rate sigmoid(v) >= 2^-125: one token from
    nothing.  The sigmoid is good to 2 |v| units of 2^-24; the factor takes half of that, the
    gates' gradients no more than all of it: 2^-16, and 2^-15 with every other rounding."""
    D, V = 64, [-60.0, -70.0, -80.0, -81.0, -82.0]
    B = len(V)
    gate = torch.tensor(V, device=DEV)[:, None, None].expand(B, 1, D).contiguous()
    rate = torch.linspace(0.02, 0.1, D, device=DEV)
    x, dy = rnd(B, 1, D, seed=1), rnd(B, 1, D, seed=2)
    s = torch.sigmoid(gate.cpu().double())
    r, xd, d = rate.cpu().double(), x.cpu().double(), dy.cpu().double()
    assert float((r * s).min()) >= 2.0 ** -125
    c = -torch.expm1(-r * s)
    k = torch.sqrt(c * (2 - c))
    y, hT = gdn.glr_forward(x, gate, rate=rate, form="rate", scale="norm")
    dx, dg, _, dr, _ = gdn.glr_backward(dy, x, gate, rate=rate, form="rate", scale="norm")
    da = -d * xd * (1 - c).square() / k
    for v, want, what in ((y, k * xd, "y"), (hT, (k * xd)[:, 0], "hT"), (dx, k * d, "dx"), (dg, -da * r * s * (1 - s), "dgate")):
        close(v, want, want.abs() * 2.0 ** -15, what)
    close(dr, -(da * s).sum((0, 1)), (da * s).abs().sum((0, 1)) * 2.0 ** -15, "drate")
    # farther: rate sigmoid(v) is a denormal number or 0, every result smaller than the root of 2^-126 times |x| or |dy| < 8
    gate = torch.tensor([-85.0, -86.0, -87.0, -88.0, -200.0], device=DEV)[:, None, None].expand(B, 1, D).contiguous()
    y, hT = gdn.glr_forward(x, gate, rate=rate, form="rate", scale="norm")
    for t in (y, hT, *gdn.glr_backward(dy, x, gate, rate=rate, form="rate", scale="norm")):
        assert t is None or (t.abs() < 2.0 ** -54).all()


@pytest.mark.parametrize("bias", [0.0, 10.0, 60.0, 300.0, 46080.0, 1474560.0])
@pytest.mark.parametrize("form", ["sigmoid", "rate", "log"])
@pytest.mark.parametrize("gt", [F32, BF])
def test_gates_that_their_bias_cancels(bias, form, gt):
    """gate + bias of ordinary size, each of them of any: final states of memories of a thousand tokens
    within 1e-6 of the recurrence's, and every value within the oracle's errors."""
    T, D = 3000, 6
    v = rnd(1, T, D, seed=1)
    v = -v.abs() / 1000 if form == "log" else v + (7 if form == "sigmoid" else 0)
    gate, b = (v - bias).to(gt), torch.full((D,), bias, device=DEV)
    if form == "log":           # (rounded, gate + bias may be above zero: growing states are another test's)
        gate = torch.where(gate.float() + bias > 0, torch.full_like(gate, -bias), gate)
    rate = torch.linspace(0.001, 0.02, D, device=DEV) if form == "rate" else None
    x, dy = rnd(1, T, D, seed=2), rnd(1, T, D, seed=3)
    x, dy = (x, dy) if gt == F32 else (x.to(BF), dy.to(BF))
    kw = dict(gate_bias=b, rate=rate, form=form, scale="complement")
    y, hT = gdn.glr_forward(x, gate, **kw)
    grads = gdn.glr_backward(dy, x, gate, **kw)
    ref = L.glr(x[0], gate[0], b, rate, None, [T], form, "complement", dy[0])
    glr_close((y, hT, *grads), ref, ("y", "hT", "dx", "dgate", "dbias", "drate"))
    assert (hT.cpu().double() - ref["hT"]).norm() <= 1e-6 * ref["hT"].norm()
    state = torch.zeros(1, D, device=DEV)
    for t in range(3):
        gdn.glr_step(x[:, t], gate[:, t], state, **kw)
    ref = L.glr(x[0, :3], gate[0, :3], b, rate, None, [3], form, "complement")
    glr_close((state,), ref, ("hT",))


def test_gradients_in_any_layout():
    """The same bits wherever they go: time-major, halves of a batch, side by side in either."""
    B, T, D = 3, 77, 64
    x, gate, dy = (rnd(B, T, D, seed=i, dtype=BF) for i in range(3))
    kw = dict(rate=torch.full((D,), 0.1, device=DEV), form="rate", scale="norm")
    want = gdn.glr_backward(dy, x, gate, **kw)
    halves, tokens = torch.empty(B, 2, T, D, device=DEV, dtype=BF), torch.empty(T, B, 2 * D, device=DEV, dtype=BF)
    for dx, dg in ((halves[:, 0], halves[:, 1]), (tokens[..., D:].transpose(0, 1), tokens[..., :D].transpose(0, 1))):
        got = gdn.glr_backward(dy, x, gate, dx=dx, dgate=dg, **kw)
        assert got[0] is dx and got[1] is dg and torch.equal(dx, want[0]) and torch.equal(dg, want[1]) and torch.equal(got[3], want[3])
