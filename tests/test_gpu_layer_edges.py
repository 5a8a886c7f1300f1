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
