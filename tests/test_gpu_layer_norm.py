"""Root-mean-square norm on the GPU against its definition in 64 bits.

Tolerances.  Statistics are sums of D squares (or products) in fp32 over at most
32 values a lane and then a tree: a relative error of at most (32 + 12) 2^-24
of the sum of the terms' sizes; r takes half of that, a division and a square
root; with the products after it every value is within 64 * 2^-24 = 2^-18 of
its terms' size, plus half a step of the type it is stored in (bf16 2^-8,
fp32 2^-24, e4m3 2^-4)."""
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


CASES = [  # rows, D, x type, residual type
    (1, 1, BF, BF), (3, 5, F32, F32), (7, 64, BF, F32), (5, 255, BF, BF), (9, 256, F32, F32), (2, 260, BF, BF),
    (6, 1023, BF, F32), (4, 1024, BF, BF), (3, 2050, F32, F32), (5, 4100, BF, BF), (2, 8192, BF, BF), (3, 8191, BF, F32),
    (2, 8200, F32, F32), (2, 16384, BF, BF), (2, 16383, BF, BF), (769, 96, BF, BF), (1600, 257, BF, F32),
    (3, 2, BF, F32), (5, 130, BF, BF), (4, 1022, F32, F32), (3, 1030, BF, BF), (3, 4098, BF, F32), (2, 8190, BF, BF),
    (2, 16382, BF, F32), (1700, 254, BF, BF)]


@pytest.mark.parametrize("rows,D,dt,rt", CASES)
def test_forward_and_backward(rows, D, dt, rt):
    x, res = rnd(rows, D, seed=1, dtype=dt), rnd(rows, D, seed=2, dtype=rt, scale=3.0)
    w = rnd(D, seed=3, dtype=F32 if D % 2 else dt) + 1.0
    w = w.to(F32 if D % 2 else dt)
    y, s, scales = gdn.norm_forward(x, w, res, eps=1e-5)
    assert scales is None and s.dtype == rt and y.dtype == dt
    assert torch.equal(s, (x.float() + res.float()).to(rt))
    ref, kept = L.norm(x, w, res, 1e-5, rt)
    close(y, ref, ref.abs() * (HALF[dt] + ARITH), "y")
    dy, dres = rnd(rows, D, seed=4, dtype=dt), rnd(rows, D, seed=5, dtype=rt)
    ds, dx, dw = gdn.norm_backward(dy, s, w, dres, eps=1e-5, x_dtype=dt)
    rs, rw = L.norm_grad(dy, kept, w, dres, 1e-5)
    # sizes of the terms of ds and dw
    r = (kept.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    u = (dy.cpu().double() * w.cpu().double()).abs()
    size = dres.cpu().double().abs() + r * (u + kept.abs() * r * r * (u * kept.abs()).mean(-1, keepdim=True))
    close(ds, rs, rs.abs() * HALF[rt] + size * ARITH, "ds")
    close(dx, rs, rs.abs() * HALF[dt] + size * ARITH, "dx")
    assert (dx is ds) == (dt == rt)
    # dw: rows / 768 of a workgroup's, then the partial sums in 64 lines
    terms = (dy.cpu().double() * kept * r).abs().sum(0)
    close(dw, rw, terms * (ARITH + (rows / 768 + 64) * 2.0 ** -24), "dw")


@pytest.mark.parametrize("rows,D", [(4, 64), (3, 130), (5, 256), (2, 1000), (3, 1001), (2, 8192), (2, 9000), (3, 1002),
                                    (2, 4098), (2, 16382)])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dt", [BF, F32])
def test_eight_bit_output(rows, D, group, dt):
    x = rnd(rows, D, seed=1, dtype=dt)
    x[0] = 0                                    # a row of zeros: the least scale, zeros
    w = (rnd(D, seed=2, scale=0.2) + 1).to(dt)
    q, s, scale = gdn.norm_forward(x, w, eps=1e-6, out_dtype=FP8, group=group)
    assert s is None and q.dtype == FP8
    ref, _ = L.norm(x, w, None, 1e-6)
    g = group or D
    n = -(-D // g)
    assert scale.shape == (rows, n)
    amax = torch.stack([ref[:, k * g:(k + 1) * g].abs().amax(1) for k in range(n)], 1)
    want = (amax / 448).clamp(min=2.0 ** -126)
    close(scale, want, want * ARITH, "scale")
    assert float(scale[0, 0]) == 2.0 ** -126 and not q[0].float().any()
    full = scale.cpu().double().repeat_interleave(g, 1)[:, :D]
    # half a step of e4m3, whose subnormals are 2^-9 apart; 448 at most
    v = ref / full
    close(q.float().cpu().double(), v, v.abs() * (2.0 ** -4 + ARITH) + 2.0 ** -10, "q")
    assert q.float().abs().max() <= 448
    # the largest of a group is the largest there is
    assert (q[1:].float().abs().amax(1) == 448).all()


def test_nan_and_infinity():
    x = rnd(4, 512, seed=1, dtype=BF)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    w = torch.ones(512, device=DEV, dtype=BF)
    y, _, _ = gdn.norm_forward(x, w)
    clean = gdn.norm_forward(x[3:], w)[0]
    assert y[1].isnan().all() and torch.equal(y[3:], clean) and y[0].isfinite().all()
    # r = 1 / inf = 0 there: zeros, and 0 * inf
    assert y[2, 9].isnan() and y[2, :9].eq(0).all()
    q, _, scale = gdn.norm_forward(x, w, out_dtype=FP8, group=128)
    assert q[1].float().isnan().all() and q[3].float().isfinite().all()
    # the groups without the infinity are zeros at the least scale
    assert float(scale[2, 1]) == 2.0 ** -126 and not q[2, 128:].float().any()


def test_strided_rows_views_and_in_place():
    big = rnd(6, 3, 512, seed=1, dtype=BF)
    w = rnd(256, seed=2, dtype=BF)
    x = big[:, 1, 128:384]
    a = gdn.norm_forward(x, w)[0]
    assert torch.equal(a, gdn.norm_forward(x.contiguous(), w)[0])
    x = big[:, 1, 129:385]                       # no longer aligned to four elements
    b = gdn.norm_forward(x, w)[0]
    ref, _ = L.norm(x, w, None, 1e-6)
    close(b, ref, ref.abs() * (2.0 ** -8 + ARITH), "unaligned")
    res = rnd(6, 256, seed=3, dtype=BF)
    y0, s0, _ = gdn.norm_forward(big[:, 0, :256], w, res)
    keep = res.clone()
    y1, s1, _ = gdn.norm_forward(big[:, 0, :256], w, res, s=res)
    assert s1 is res and torch.equal(res, s0) and torch.equal(y0, y1) and not torch.equal(res, keep)
    d = rnd(6, 256, seed=4, dtype=BF)
    ds0, _, dw0 = gdn.norm_backward(y0, s0, w, d)
    ds1, _, dw1 = gdn.norm_backward(y0, s0, w, d, ds=d)
    assert ds1 is d and torch.equal(ds0, ds1) and torch.equal(dw0, dw1)


def test_empty_and_refused():
    w = torch.ones(64, device=DEV)
    y, s, _ = gdn.norm_forward(torch.empty(0, 64, device=DEV), w, torch.empty(0, 64, device=DEV))
    assert y.shape == s.shape == (0, 64)
    ds, dx, dw = gdn.norm_backward(y, s, w)
    assert dw.eq(0).all() and ds.shape == (0, 64)
    x = rnd(4, 64, seed=1)
    for bad, err in ((lambda: gdn.norm_forward(x, w[:32]), ValueError), (lambda: gdn.norm_forward(x.half(), w), TypeError),
                     (lambda: gdn.norm_forward(x, w, out_dtype=BF), TypeError), (lambda: gdn.norm_forward(x, w, group=32), ValueError),
                     (lambda: gdn.norm_forward(x.T, w[:4]), ValueError), (lambda: gdn.norm_forward(x, w, y=x), ValueError),
                     (lambda: gdn.norm_forward(x, w, x.cpu()), ValueError),
                     (lambda: gdn.norm_forward(rnd(1, 16388, seed=1), rnd(16388, seed=1)), gdn.GdnError),
                     (lambda: gdn.norm_backward(x, x.to(BF), w), TypeError),
                     (lambda: gdn.norm_forward(x, w, eps=-1.0), gdn.GdnError)):
        with pytest.raises(err):
            bad()


def test_more_rows_than_a_launch_takes():
    rows, D = (1 << 22) + 5, 8
    x, res = rnd(rows, D, seed=1, dtype=BF), rnd(rows, D, seed=2, dtype=BF)
    w = rnd(D, seed=3) + 1.0
    y, s, _ = gdn.norm_forward(x, w, res)
    q, t, scales = gdn.norm_forward(x, w, res, out_dtype=torch.float8_e4m3fn, group=128)
    # each row is its own: those of a second launch and of the first are what
    # they are among few
    for at in (slice(0, 64), slice((1 << 22) - 3, rows)):
        a, b, _ = gdn.norm_forward(x[at], w, res[at])
        assert torch.equal(y[at], a) and torch.equal(s[at], b) and torch.equal(t[at], b)
        a, _, b = gdn.norm_forward(x[at], w, res[at], out_dtype=torch.float8_e4m3fn, group=128)
        assert torch.equal(q[at].view(torch.uint8), a.view(torch.uint8)) and torch.equal(scales[at], b)


def test_overlapping_arguments_refused():
    x, w = rnd(4, 64, seed=1), torch.ones(64, device=DEV)
    with pytest.raises(ValueError):                 # every second element of a buffer
        gdn.norm_forward(rnd(128, seed=1)[::2], w)
    with pytest.raises(ValueError):                 # s may be the residual, but not x too
        gdn.norm_forward(x, w, x, s=x)
    with pytest.raises(ValueError):                 # ds may be dres, but not dy too
        gdn.norm_backward(x, x + 1, w, x, ds=x)


def test_gradient_against_differences():
    """fp32 along a direction: the loss, summed in 64 bits from fp32 outputs, is
    known to 2^-18 of its terms (see above), a difference over 2 * 2^-8 so to
    2^-10 of them, and differs from the derivative by the cube's term, below
    (2^-8)^2 of the terms' sizes times a few."""
    R, D, h = 8, 512, 2.0 ** -8
    x, res, w, dy = (rnd(*s, seed=i) for i, s in enumerate(((R, D), (R, D), (D,), (R, D))))
    dres = rnd(R, D, seed=9)

    def loss(x, w):
        y, s, _ = gdn.norm_forward(x, w, res, eps=1e-2)
        return (y.double() * dy.double()).sum() + (s.double() * dres.double()).sum()

    _, s, _ = gdn.norm_forward(x, w, res, eps=1e-2)
    ds, _, dw = gdn.norm_backward(dy, s, w, dres, eps=1e-2)
    for n, (g, at) in enumerate(((ds, x), (dw, w))):
        d = rnd(*at.shape, seed=20 + n)
        args = [(x + h * d, w), (x - h * d, w)] if n == 0 else [(x, w + h * d), (x, w - h * d)]
        num = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        terms = float((dy.abs() * w.abs()).double().sum() + dres.abs().double().sum())
        assert abs(float(num - (g.double() * d.double()).sum())) <= terms * 2.0 ** -9, n


def test_streams_graphs_and_repeats():
    x, res, w, dy = rnd(300, 2048, seed=1, dtype=BF), rnd(300, 2048, seed=2, dtype=BF), rnd(2048, seed=3, dtype=BF), rnd(300, 2048, seed=4, dtype=BF)

    def work():
        y, s, _ = gdn.norm_forward(x, w, res)
        q, _, sc = gdn.norm_forward(x, w, res, out_dtype=FP8, group=128)
        return [y, s, q.view(torch.uint8), sc, *gdn.norm_backward(dy, s, w, res)]

    ref = [t.clone() for t in work()]
    assert all(torch.equal(a, b) for a, b in zip(ref, work()))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, s, _ = gdn.norm_forward(x, w, res, stream=st)
    st.synchronize()
    assert torch.equal(y, ref[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        x.copy_(rnd(300, 2048, seed=10 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, work())), k


@pytest.mark.parametrize("D,group", [(64, 0), (256, 0), (1024, 128), (4096, 0), (8192, 128), (16384, 128)])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_eight_bit_ties_are_those_of_the_quotient(D, group, at):
    """Rows of ones: r = 1 and y is the weight itself, so the stored values are e4m3 of
    weight / scale, bit for bit.  The weights lie at halfway points times the scale,
    where a product with 1 / scale rounds to the other side now and then."""
    g = torch.Generator().manual_seed(D + at)
    n = group or D
    amax = torch.rand(D // n, generator=g) * 6 + 1
    scale = amax / 448
    tie = (torch.randint(8, 16, (D // n, n), generator=g) + 0.5) * 2.0 ** torch.randint(-8, 5, (D // n, n), generator=g).float()
    w = tie * scale[:, None] * torch.where(torch.rand(D // n, n, generator=g) < 0.5, -1.0, 1.0)
    w[:, 0] = amax
    want = (w / scale[:, None]).to(FP8).reshape(-1)
    # (the weight's alignment chooses how many elements a lane takes)
    weight = torch.empty(D + at, device=DEV)[at:].copy_(w.reshape(-1))
    q, _, s = gdn.norm_forward(torch.ones(3, D, device=DEV), weight, eps=0.0, out_dtype=FP8, group=group)
    assert torch.equal(s.cpu(), scale.reshape(1, -1).expand(3, -1))
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8).expand(3, -1))


def test_eight_bit_rows_with_infinite_values():
    """An infinite weight: the largest value is infinite, its quotient no number, and
    every finite value over the infinite scale zero."""
    x = torch.ones(2, 256, device=DEV)
    w = torch.full((256,), 2.0, device=DEV)
    w[200] = float("inf")
    for group in (0, 128):
        q, _, scale = gdn.norm_forward(x, w, eps=0.0, out_dtype=FP8, group=group)
        hit = slice(128 if group else 0, 256)
        f = q.float()
        assert f[:, 200].isnan().all() and scale[:, -1].isinf().all()
        rest = torch.cat([f[:, hit][:, :200 - hit.start], f[:, 201:]], 1)
        assert rest.eq(0).all()
        if group:
            assert f[:, :128].eq(448).all() and scale[:, 0].eq(2.0 / 448).all()
