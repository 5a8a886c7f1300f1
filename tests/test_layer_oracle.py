"""The layer oracle's gradients against finite differences of its forward forms
(64 bits, CPU), and its forward forms against other ways to the same numbers."""
import pytest

torch = pytest.importorskip("torch")

from oracle import layer as L

EPS = 1e-6


def rnd(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def differences(f, leaves, grads, seed=0):
    """Each gradient along a direction against central differences.  With steps
    of 1e-5 in 64 bits the two agree to a few 1e-9 of the terms' size."""
    for i, (x, g) in enumerate(zip(leaves, grads)):
        d = rnd(*x.shape, seed=seed + 100 + i)
        plus, minus = list(leaves), list(leaves)
        plus[i], minus[i] = x + EPS * d, x - EPS * d
        num = (f(*plus) - f(*minus)) / (2 * EPS)
        ana = (g * d).sum()
        assert abs(num - ana) <= 1e-6 * (1 + (g * d).abs().sum()), (i, float(num), float(ana))


def test_norm_grad():
    x, w, r, dy, dres = rnd(5, 33, seed=1), rnd(33, seed=2), rnd(5, 33, seed=3), rnd(5, 33, seed=4), rnd(5, 33, seed=5)

    def loss(x, w, r):
        s = x + r
        y = s * (s.square().mean(-1, keepdim=True) + 1e-3).rsqrt() * w
        return (y * dy).sum() + (s * dres).sum()

    ds, dw = L.norm_grad(dy, x + r, w, dres, 1e-3)
    differences(loss, (x, w, r), (ds, dw, ds))


@pytest.mark.parametrize("silu", [False, True])
def test_conv_grad(silu):
    lens = [4, 0, 1, 7]
    D, W = 6, 4
    x, w, b, st = rnd(12, D, seed=1), rnd(D, W, seed=2), rnd(D, seed=3), rnd(4, W - 1, D, seed=4)
    dy, df = rnd(12, D, seed=5), rnd(4, W - 1, D, seed=6)

    def loss(x, w, b, st):
        y, last = L.conv(x, w, b, st, lens, silu)
        return (y * dy).sum() + (last * df).sum()

    dx, dw, db, ds = L.conv_grad(dy, x, w, b, st, lens, silu, df)
    differences(loss, (x, w, b, st), (dx, dw, db, ds))


def test_conv_is_a_grouped_convolution():
    x, w, b = rnd(9, 5, seed=1), rnd(5, 3, seed=2), rnd(5, seed=3)
    y, last = L.conv(x, w, b, None, [9], False)
    ref = torch.nn.functional.conv1d(x.T[None], w[:, None], b, padding=2, groups=5)[0, :, :9].T
    assert torch.allclose(y, ref, rtol=1e-13, atol=1e-13)
    assert torch.equal(last[0], x[-2:])


def test_ssm_grad():
    lens = [5, 0, 1, 6]
    T, H, P, N, G = 12, 4, 3, 5, 2
    x, dt, A = rnd(T, H, P, seed=1), rnd(T, H, seed=2).exp() * 0.3, -rnd(H, seed=3).exp()
    B, C, D, h0 = rnd(T, G, N, seed=4), rnd(T, G, N, seed=5), rnd(H, seed=6), rnd(4, H, N, P, seed=7)
    dy, dhT = rnd(T, H, P, seed=8), rnd(4, H, N, P, seed=9)

    def loss(x, dt, A, B, C, D, h0):
        y, hT = L.ssm(x, dt, A, B, C, D, h0, lens)
        return (y * dy).sum() + (hT * dhT).sum()

    g = L.ssm_grad(dy, x, dt, A, B, C, D, h0, lens, dhT)
    differences(loss, (x, dt, A, B, C, D, h0), [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")])


def test_ssm_is_the_recurrence_of_the_gated_oracle_without_erasure():
    """One head with one-hot, orthogonal keys: the delta rule erases nothing
    there, so the gated oracle and this one agree (q = C, k = B, v = dt x with
    beta 1, g = dt A)."""
    import numpy as np
    import oracle
    T, P, N = 6, 4, 8
    x, dt, A = rnd(T, 1, P, seed=1), rnd(T, 1, seed=2).exp() * 0.1, torch.tensor([-2.0], dtype=torch.float64)
    B = torch.eye(N, dtype=torch.float64)[:T][:, None]
    C = rnd(T, 1, N, seed=3)
    y, hT = L.ssm(x, dt, A, B, C, None, None, [T])
    n = lambda t: t[None].numpy()  # noqa: E731
    o, h = oracle.token_recurrence(n(C), n(B), n(x * dt[..., None]), np.ones((1, T, 1)), n(dt * A), None)
    # the gated oracle reads 32-bit inputs: v, g and C are rounded by 2^-24, a
    # decay over six tokens by six times |g| < 2 of that, values stay below 4
    assert np.allclose(o[0], y.numpy(), rtol=0, atol=64 * 2.0 ** -24) and np.allclose(h[0], hT[0].numpy(), rtol=0, atol=64 * 2.0 ** -24)
