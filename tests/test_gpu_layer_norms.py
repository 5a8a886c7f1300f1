"""Layer norm and the gated norm on the GPU against their definitions in 64 bits.

Tolerances.  A row's sums are of at most 32 values a lane and then a tree, 44
roundings of 2^-24 of the terms' sizes; a mean is taken out to 44 2^-24 of the row's
mean size behind it, a deviation or less; r takes half of the squares' error, a
division and a square root; the gate's sigmoid is within 8 2^-24.  So every value is
within 64 * 2^-24 = 2^-18 of its terms' sizes (the oracle's, where a centred
value's size is |h| + 1), plus half a step of the type it is stored in (bf16
2^-8, fp32 2^-24, e4m3 2^-4)."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ARITH = 2.0 ** -18


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def close(got, ref, tol, what):
    d = (got.detach().cpu().double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e over its tolerance" % (what, int(bad.sum()), bad.numel(),
                                                                               float((d - tol).max()))


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

LN_CASES = [  # rows, D, x type, residual type, bias
    (1, 1, BF, BF, True), (3, 5, F32, F32, False), (7, 64, BF, F32, True), (5, 255, BF, BF, True), (9, 256, F32, F32, True),
    (2, 260, BF, BF, False), (6, 1023, BF, F32, True), (4, 1024, BF, BF, True), (3, 2050, F32, F32, True), (5, 4100, BF, BF, True),
    (2, 8192, BF, BF, True), (3, 8191, BF, F32, True), (2, 8200, F32, F32, True), (2, 16384, BF, BF, True), (2, 16383, BF, BF, False),
    (513, 96, BF, BF, True), (1600, 257, BF, F32, True), (3, 2, BF, F32, True), (5, 130, BF, BF, True), (4, 1022, F32, F32, True),
    (3, 4098, BF, F32, True), (2, 8190, BF, BF, True), (2, 16382, BF, F32, True), (1700, 254, BF, BF, True), (1030, 520, F32, F32, True)]


@pytest.mark.parametrize("rows,D,dt,rt,bias", LN_CASES)
def test_layer_norm_forward_and_backward(rows, D, dt, rt, bias):
    x, res = rnd(rows, D, seed=1, dtype=dt), rnd(rows, D, seed=2, dtype=rt, scale=3.0) + 2.0
    res = res.to(rt)
    wt = F32 if D % 2 else dt
    w, b = (rnd(D, seed=3) + 1.0).to(wt), rnd(D, seed=6, dtype=wt) if bias else None
    y, s, scales = gdn.layer_norm_forward(x, w, b, res, eps=1e-3)
    assert scales is None and s.dtype == rt and y.dtype == dt
    assert torch.equal(s, (x.float() + res.float()).to(rt))
    ref, kept, h = L.layer_norm(x, w, b, res, 1e-3, rt)
    wd = w.cpu().double().abs()
    size = (h.abs() + 1) * wd + (0 if b is None else b.cpu().double().abs())
    close(y, ref, ref.abs() * HALF[dt] + size * ARITH, "y")
    dy, dres = rnd(rows, D, seed=4, dtype=dt), rnd(rows, D, seed=5, dtype=rt)
    ds, dx, dw, db = gdn.layer_norm_backward(dy, s, w, b, dres, eps=1e-3, x_dtype=dt)
    rs, rw, rb = L.layer_norm_grad(dy, kept, w, dres, 1e-3)
    v = kept - kept.mean(-1, keepdim=True)
    r = (v.square().mean(-1, keepdim=True) + 1e-3).rsqrt()
    u, hs = dy.cpu().double().abs() * wd, h.abs() + 1
    size = dres.cpu().double().abs() + r * (u + u.mean(-1, keepdim=True) + hs * (u * hs).mean(-1, keepdim=True))
    close(ds, rs, rs.abs() * HALF[rt] + size * ARITH, "ds")
    close(dx, rs, rs.abs() * HALF[dt] + size * ARITH, "dx")
    assert (dx is ds) == (dt == rt) and (db is None) == (b is None)
    # rows / 512 of a workgroup's, then the partial sums in 64 lines
    many = (rows / 512 + 64) * 2.0 ** -24
    d = dy.cpu().double().abs()
    close(dw, rw, (d * hs).sum(0) * (ARITH + many), "dw")
    if b is not None:
        close(db, rb, d.sum(0) * (many + 2.0 ** -23), "db")


def test_rows_far_from_zero_keep_their_digits():
    """Rows of 4096 + n / 8: sums of squares first would leave nothing.  The values are
    exact in fp32, so only the arithmetic's errors remain."""
    x = (4096 + torch.randint(-8, 9, (5, 1000), generator=torch.Generator().manual_seed(1)).float() / 8).to(DEV)
    w, b = rnd(1000, seed=2), rnd(1000, seed=3)
    y, _, _ = gdn.layer_norm_forward(x, w, b)
    ref, _, h = L.layer_norm(x, w, b, None, 1e-5)
    close(y, ref, (h.abs() + 1) * w.cpu().double().abs() * ARITH + b.cpu().double().abs() * ARITH, "y")
    # equal elements: y is the bias
    y, _, _ = gdn.layer_norm_forward(torch.full((2, 1000), 4097.3, device=DEV), w, b)
    # (a mean's error, 44 2^-24 of 4097, is taken out to 44 2^-24 of itself; over sqrt(eps) 9e-6 is left)
    assert (y - b).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("rows,D", [(4, 64), (3, 130), (5, 256), (2, 1000), (3, 1001), (2, 8192), (2, 9000), (3, 1002),
                                    (2, 4098), (2, 16382)])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dt", [BF, F32])
def test_layer_norm_eight_bit_output(rows, D, group, dt):
    x = rnd(rows, D, seed=1, dtype=dt)
    x[0] = 0                                    # zeros and no bias: the least scale, zeros
    w = (rnd(D, seed=2, scale=0.2) + 1).to(dt)
    q, s, scale = gdn.layer_norm_forward(x, w, out_dtype=FP8, group=group)
    assert s is None and q.dtype == FP8
    ref, _, h = L.layer_norm(x, w, None, None, 1e-5)
    g = group or D
    n = -(-D // g)
    assert scale.shape == (rows, n)
    size = (h.abs() + 1) * w.cpu().double().abs() * ARITH
    amax = torch.stack([ref[:, k * g:(k + 1) * g].abs().amax(1) for k in range(n)], 1)
    slack = torch.stack([size[:, k * g:(k + 1) * g].amax(1) for k in range(n)], 1) / 448
    want = (amax / 448).clamp(min=2.0 ** -126)
    close(scale, want, want * ARITH + slack, "scale")
    assert float(scale[0, 0]) == 2.0 ** -126 and not q[0].float().any()
    full = scale.cpu().double().repeat_interleave(g, 1)[:, :D]
    v = ref[1:] / full[1:]
    # half a step of e4m3, whose subnormals are 2^-9 apart; 448 at most
    close(q[1:].float().cpu().double(), v, v.abs() * (2.0 ** -4 + ARITH) + 2.0 ** -10 + size[1:] / full[1:], "q")
    assert q.float().abs().max() <= 448


def test_layer_norm_nan_infinity_and_strides():
    x = rnd(4, 512, seed=1, dtype=BF)
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    w, b = torch.ones(512, device=DEV, dtype=BF), rnd(512, seed=2, dtype=BF)
    y, _, _ = gdn.layer_norm_forward(x, w, b)
    assert y[1:3].isnan().all() and y[0].isfinite().all() and torch.equal(y[3:], gdn.layer_norm_forward(x[3:], w, b)[0])
    ds, _, _, _ = gdn.layer_norm_backward(y, x, w, b)
    assert ds[1:3].isnan().all() and ds[0].isfinite().all() and ds[3].isfinite().all()
    big = rnd(6, 3, 512, seed=1, dtype=BF)
    w, b = rnd(256, seed=2, dtype=BF), rnd(256, seed=3, dtype=BF)
    for first in (128, 130, 129):               # aligned to four elements, two, one
        v = big[:, 1, first:first + 256]
        ref, _, h = L.layer_norm(v, w, b, None, 1e-5)
        close(gdn.layer_norm_forward(v, w, b)[0], ref, ref.abs() * HALF[BF] + ((h.abs() + 1) * w.cpu().double().abs() + 1) * ARITH, first)
    res = rnd(6, 256, seed=3, dtype=BF)
    y0, s0, _ = gdn.layer_norm_forward(big[:, 0, :256], w, b, res)
    y1, s1, _ = gdn.layer_norm_forward(big[:, 0, :256], w, b, res, s=res)
    assert s1 is res and torch.equal(res, s0) and torch.equal(y0, y1)
    d = rnd(6, 256, seed=4, dtype=BF)
    a0 = gdn.layer_norm_backward(y0, s0, w, b, d)
    a1 = gdn.layer_norm_backward(y0, s0, w, b, d, ds=d)
    assert a1[0] is d and all(torch.equal(p, q) for p, q in zip(a0, a1))


def test_layer_norm_empty_and_many_rows():
    w = torch.ones(64, device=DEV)
    y, s, _ = gdn.layer_norm_forward(torch.empty(0, 64, device=DEV), w, w, torch.empty(0, 64, device=DEV))
    ds, _, dw, db = gdn.layer_norm_backward(y, s, w, w)
    assert y.shape == ds.shape == (0, 64) and dw.eq(0).all() and db.eq(0).all()
    rows, D = (1 << 22) + 5, 8
    x, w = rnd(rows, D, seed=1, dtype=BF), rnd(D, seed=3) + 1.0
    y, _, _ = gdn.layer_norm_forward(x, w)
    for at in (slice(0, 64), slice((1 << 22) - 3, rows)):
        assert torch.equal(y[at], gdn.layer_norm_forward(x[at], w)[0])


# ---------------------------------------------------------------------------
# gated norm
# ---------------------------------------------------------------------------

GN_CASES = [  # T, H, D, type, act, gate first, centred, weights of each head
    (1, 1, 1, BF, "silu", False, False, False), (5, 3, 64, BF, "silu", False, False, False), (37, 2, 128, BF, "silu", False, False, True),
    (9, 4, 128, F32, "sigmoid", False, True, False), (3, 2, 100, BF, "silu", True, False, True), (4, 3, 65, F32, "silu", False, True, True),
    (2, 5, 256, BF, "sigmoid", True, True, True), (3, 2, 250, BF, "silu", True, False, False), (4, 1, 512, F32, "silu", True, False, False),
    (3, 2, 511, BF, "silu", False, True, True), (2, 2, 1024, BF, "silu", True, False, True), (5, 2, 1000, F32, "silu", False, False, False),
    (2, 2, 1023, F32, "sigmoid", True, True, True), (3, 1, 2048, BF, "silu", True, False, True), (2, 1, 2047, BF, "silu", False, True, False),
    (2, 2, 4096, F32, "silu", True, False, True), (2, 1, 4095, BF, "silu", True, True, False), (3, 1, 8192, BF, "silu", True, False, False),
    (2, 1, 8191, F32, "silu", False, True, False), (2, 1, 8188, F32, "silu", True, True, True), (700, 16, 64, BF, "silu", False, False, False),
    (900, 9, 32, BF, "silu", False, True, True), (2100, 1, 300, BF, "silu", True, False, True), (1500, 3, 7, F32, "silu", False, True, True)]


@pytest.mark.parametrize("T,H,D,dt,act,first,center,each", GN_CASES)
def test_gate_norm_forward_and_backward(T, H, D, dt, act, first, center, each):
    x, dy = rnd(T, H, D, seed=1, dtype=dt), rnd(T, H, D, seed=2, dtype=dt)
    z = rnd(T, (H + 1) * D, seed=3, dtype=dt, scale=2.0)[:, D:].unflatten(-1, (H, D))       # a part of a projection's rows
    wt = F32 if D % 2 else dt
    shape = (H, D) if each and H > 0 else (D,)
    w, b = (rnd(*shape, seed=4) + 1.0).to(wt), rnd(*shape, seed=5, dtype=wt) if center else None
    kw = dict(eps=1e-3, activation=act, gate_first=first, center=center)
    y = gdn.gate_norm_forward(x, z, w, b, **kw)
    assert y.dtype == dt and y.is_contiguous()
    ref = L.gate_norm(x, z, w, b, 1e-3, act, first, center, dy)
    close(y, ref["y"], ref["y"].abs() * HALF[dt] + ref["ysize"] * ARITH, "y")
    dz = torch.empty(T, (H + 1) * D, device=DEV, dtype=dt).fill_(7.0)
    dx, got, dw, db = gdn.gate_norm_backward(dy, x, z, w, b, dz=dz[:, D:].unflatten(-1, (H, D)), **kw)
    assert dz[:, :D].eq(7.0).all()
    close(dx, ref["dx"], ref["dx"].abs() * HALF[dt] + ref["dxsize"] * ARITH, "dx")
    close(got, ref["dz"], ref["dz"].abs() * HALF[dt] + ref["dzsize"] * ARITH, "dz")
    # of a class's at most 1024 workgroups one row's slot after the other, 16 slots, then 64 lines
    rows = T if each else T * H
    many = (rows / 64 + 16 + 64 + 16) * 2.0 ** -24
    for name, v in (("dw", dw), ("db", db)):
        assert (v is None) == (name == "db" and not center)
        if v is not None:
            r, size = (ref[name], ref[name + "size"]) if each else (ref[name].sum(0), ref[name + "size"].sum(0))
            close(v, r, size * (ARITH + many), name)
    again = gdn.gate_norm_backward(dy, x, z, w, b, **kw)
    assert torch.equal(again[0], dx) and torch.equal(again[1], got) and torch.equal(again[2], dw)


def test_gate_norm_layouts():
    """Tokens and heads at strides of their own, in any order, and rows of two dimensions."""
    T, H, D = 6, 4, 64
    w = rnd(D, seed=2, dtype=BF)
    x, z = rnd(T, H, D, seed=1, dtype=BF), rnd(T, H, D, seed=3, dtype=BF)
    want = gdn.gate_norm_forward(x, z, w)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(gdn.gate_norm_forward(heads_first, z, w), want)
    odd = torch.empty(T, H, D + 1, device=DEV, dtype=BF)[..., 1:]
    odd.copy_(z)
    unaligned = gdn.gate_norm_forward(x, odd, w)
    ref = L.gate_norm(x, z, w, None, 1e-5, "silu", False, False)
    close(unaligned, ref["y"], ref["y"].abs() * HALF[BF] + ref["ysize"] * ARITH, "unaligned")
    assert torch.equal(gdn.gate_norm_forward(x.flatten(0, 1), z.flatten(0, 1), w), want.flatten(0, 1))
    assert torch.equal(gdn.gate_norm_forward(x[None], z[None], w), want[None])
    assert torch.equal(gdn.gate_norm_forward(x.unflatten(0, (2, 3)), z.unflatten(0, (2, 3)), w), want.unflatten(0, (2, 3)))
    assert torch.equal(gdn.gate_norm_forward(x[:, :1], z[:, :1], w), want[:, :1])
    assert torch.equal(gdn.gate_norm_forward(x[::2], z[::2], w), want[::2])
    assert torch.equal(gdn.gate_norm_forward(x[0, 0], z[0, 0], w), want[0, 0])
    same = z[:1].expand(T, H, D)                # one gate for all tokens
    assert torch.equal(gdn.gate_norm_forward(x, same, w), gdn.gate_norm_forward(x, same.contiguous(), w))
    dz = torch.empty(H, T, D, device=DEV, dtype=BF).transpose(0, 1)
    dx, got, dw, _ = gdn.gate_norm_backward(want, x, z, w, dz=dz)
    dx1, dz1, dw1, _ = gdn.gate_norm_backward(want, x, z, w)
    assert torch.equal(got, dz1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_gate_norm_extreme_gates_and_empty():
    x, w = rnd(8, 2, 64, seed=1), torch.ones(64, device=DEV)
    z = torch.empty(8, 2, 64, device=DEV)
    z[:] = torch.tensor([-200.0, -88.0, -30.0, -1e-30, 0.0, 30.0, 88.0, 200.0], device=DEV)[:, None, None]
    dy = rnd(8, 2, 64, seed=2)
    for act in ("silu", "sigmoid"):
        ref = L.gate_norm(x, z, w, None, 1e-5, act, False, False, dy)
        # an exponential below 2^-126, fp32's least normal number, may be zero: 2^-126 times
        # |z| < 2^7 (where it is below), |h| <= sqrt(64) = 2^3 and |dy| < 2^3
        assert float(dy.abs().max()) < 8
        tiny = 2.0 ** (-126 + 7 + 3 + 3)
        close(gdn.gate_norm_forward(x, z, w, activation=act), ref["y"], ref["ysize"] * ARITH + tiny, "y")
        dx, dz, dw, _ = gdn.gate_norm_backward(dy, x, z, w, activation=act)
        close(dx, ref["dx"], ref["dxsize"] * ARITH + tiny, "dx")
        close(dz, ref["dz"], ref["dzsize"] * ARITH + tiny, "dz")
    x[3, 1, 5] = float("nan")
    y = gdn.gate_norm_forward(x, z, w)
    assert y[3, 1].isnan().all() and y[3, 0].isfinite().all() and y[4].isfinite().all()
    e = torch.empty(0, 2, 64, device=DEV)
    dx, dz, dw, _ = gdn.gate_norm_backward(e, e, e, w)
    assert gdn.gate_norm_forward(e, e, w).shape == dx.shape == dz.shape == (0, 2, 64) and dw.eq(0).all()


def test_gate_norm_many_rows():
    T, H, D = (1 << 21) + 3, 2, 8
    x, z, w = rnd(T, H, D, seed=1, dtype=BF), rnd(T, H, D, seed=2, dtype=BF), rnd(2, D, seed=3) + 1.0
    y = gdn.gate_norm_forward(x, z, w)
    for at in (slice(0, 64), slice((1 << 21) - 3, T)):
        assert torch.equal(y[at], gdn.gate_norm_forward(x[at], z[at], w))


def test_gradients_against_differences():
    """fp32 along a direction: losses are known to 2^-18 of their terms, a difference over
    2 * 2^-8 so to 2^-10 of them, and differs from the derivative by the cube's term, below
    (2^-8)^2 of the terms' sizes times a few tens."""
    R, H, D, h = 4, 2, 256, 2.0 ** -8
    x, z, dy = (rnd(R, H, D, seed=i) for i in range(3))
    w, b = rnd(H, D, seed=4), rnd(H, D, seed=5)
    for first in (False, True):
        kw = dict(eps=1e-2, gate_first=first, center=True)
        grads = gdn.gate_norm_backward(dy, x, z, w, b, **kw)
        args = [x, z, w, b]
        terms = float((dy.abs() * (w.abs() * 3 + b.abs()) * (1 + z.abs())).double().sum())
        for n, g in enumerate(grads):
            d = rnd(*args[n].shape, seed=20 + n)
            side = [(gdn.gate_norm_forward(*[a + s * h * d if i == n else a for i, a in enumerate(args)], **kw).double()
                     * dy.double()).sum() for s in (1, -1)]
            assert abs(float((side[0] - side[1]) / (2 * h) - (g.double() * d.double()).sum())) <= terms * 2.0 ** -9, (first, n)
    x, dy, dres, w, b = x[:, 0].contiguous(), dy[:, 0].contiguous(), rnd(R, D, seed=9), w[0].contiguous(), b[0].contiguous()
    res = rnd(R, D, seed=10)
    _, s, _ = gdn.layer_norm_forward(x, w, b, res, eps=1e-2)
    ds, _, dw, db = gdn.layer_norm_backward(dy, s, w, b, dres, eps=1e-2)
    args = [x, w, b]
    terms = float((dy.abs() * (w.abs() * 3 + b.abs())).double().sum() + dres.abs().double().sum())
    for n, g in enumerate((ds, dw, db)):
        d = rnd(*args[n].shape, seed=30 + n)

        def loss(sign):
            y, s, _ = gdn.layer_norm_forward(*[a + sign * h * d if i == n else a for i, a in enumerate(args)], res, eps=1e-2)
            return (y.double() * dy.double()).sum() + (s.double() * dres.double()).sum()

        assert abs(float((loss(1) - loss(-1)) / (2 * h) - (g.double() * d.double()).sum())) <= terms * 2.0 ** -9, n


def test_refusals():
    x, w = rnd(4, 2, 64, seed=1), torch.ones(64, device=DEV)
    wide = torch.empty(4, 2, 128, device=DEV)
    for bad, err in ((lambda: gdn.layer_norm_forward(x, w[:32]), ValueError), (lambda: gdn.layer_norm_forward(x.half(), w), TypeError),
                     (lambda: gdn.layer_norm_forward(x, w, w.to(BF)), TypeError), (lambda: gdn.layer_norm_forward(x, w, out_dtype=BF), TypeError),
                     (lambda: gdn.layer_norm_forward(x, w, group=64), ValueError), (lambda: gdn.layer_norm_forward(x, w, y=x), ValueError),
                     (lambda: gdn.layer_norm_forward(x, w, s=x), ValueError), (lambda: gdn.layer_norm_forward(x, w, eps=-1.0), gdn.GdnError),
                     (lambda: gdn.layer_norm_forward(rnd(1, 16388, seed=1), rnd(16388, seed=1)), gdn.GdnError),
                     (lambda: gdn.layer_norm_backward(x, x, w, dbias=w), ValueError), (lambda: gdn.layer_norm_backward(x, x.to(BF), w), TypeError),
                     (lambda: gdn.gate_norm_forward(x, x[:3], w), ValueError), (lambda: gdn.gate_norm_forward(x, x, w, w), ValueError),
                     (lambda: gdn.gate_norm_forward(x, x.to(BF), w), TypeError), (lambda: gdn.gate_norm_forward(x, x, w, activation="relu"), ValueError),
                     (lambda: gdn.gate_norm_forward(x[0], x[0], rnd(2, 64, seed=1)), ValueError),
                     (lambda: gdn.gate_norm_forward(x, x, rnd(3, 64, seed=1)), ValueError), (lambda: gdn.gate_norm_forward(x, x, w, y=x), ValueError),
                     (lambda: gdn.gate_norm_forward(x, x, w, eps=float("nan")), gdn.GdnError),
                     (lambda: gdn.gate_norm_forward(wide[..., ::2], x, w), ValueError),
                     (lambda: gdn.gate_norm_forward(rnd(1, 1, 8196, seed=1), rnd(1, 1, 8196, seed=1), rnd(8196, seed=1)), gdn.GdnError),
                     (lambda: gdn.gate_norm_backward(x, x, x, w, dbias=w), ValueError), (lambda: gdn.gate_norm_backward(x, x, x, w, dz=x), ValueError),
                     (lambda: gdn.gate_norm_backward(x, x, x, w, dz=torch.empty(1, 2, 64, device=DEV).expand(4, 2, 64)), ValueError)):
        with pytest.raises(err):
            bad()


def test_streams_graphs_and_repeats():
    x, z, dy = (rnd(300, 8, 128, seed=i, dtype=BF) for i in range(3))
    w, b = rnd(8, 128, seed=4, dtype=BF), rnd(1024, seed=5, dtype=BF)
    rows, res = x.flatten(1), rnd(300, 1024, seed=6, dtype=BF)

    def work():
        y = gdn.gate_norm_forward(x, z, w)
        n, s, _ = gdn.layer_norm_forward(rows, b, b, res)
        q, _, sc = gdn.layer_norm_forward(rows, b, b, res, out_dtype=FP8, group=128)
        return [y, n, s, q.view(torch.uint8), sc, *gdn.gate_norm_backward(dy, x, z, w)[:3], *gdn.layer_norm_backward(dy.flatten(1), s, b, b, res)]

    ref = [t.clone() for t in work()]
    assert all(torch.equal(a, c) for a, c in zip(ref, work()))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = gdn.gate_norm_forward(x, z, w, stream=st)
    n, _, _ = gdn.layer_norm_forward(rows, b, b, res, stream=st)
    st.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(n, ref[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        x.copy_(rnd(300, 8, 128, seed=10 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, work())), k
