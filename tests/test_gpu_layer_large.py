"""The layer norm, gated norm and gated linear recurrence at sizes whose launches, rows or
offsets pass 32 bits, against the definitions in 64 bits at some places of them."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ARITH = 2.0 ** -18          # of a row's terms, as in test_gpu_layer_norms.py


def normal(*shape, seed, dtype=BF):
    return torch.empty(*shape, device=DEV, dtype=dtype).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def close(got, ref, tol, what):
    d = (got.detach().cpu().double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e over its tolerance" % (what, int(bad.sum()), bad.numel(),
                                                                               float((d - tol).max()))


def test_gate_norm_sums_of_many_wide_heads():
    """2^25 weights and as many biases: the sums take two launches, whose border is among
    the heads compared (each is summed on its own: two rows, so one addition)."""
    T, H, D = 2, 4096, 8192
    x, z, dy = (normal(T, H, D, seed=i) for i in range(3))
    w, b = normal(H, D, seed=4), normal(H, D, seed=5)
    dx, dz, dw, db = gdn.gate_norm_backward(dy, x, z, w, b, center=True)
    at = [0, 1, 2047, H - 3, H - 2, H - 1]
    ref = L.gate_norm(x[:, at], z[:, at], w[at], b[at], 1e-5, "silu", False, True, dy[:, at])
    close(dx[:, at], ref["dx"], ref["dx"].abs() * HALF[BF] + ref["dxsize"] * ARITH, "dx")
    close(dz[:, at], ref["dz"], ref["dz"].abs() * HALF[BF] + ref["dzsize"] * ARITH, "dz")
    close(dw[at], ref["dw"], ref["dwsize"] * ARITH, "dw")
    close(db[at], ref["db"], ref["dbsize"] * ARITH, "db")
    assert db[:, ::97].any(1).all() and dw[:, ::97].any(1).all()


def test_gradients_of_very_many_short_sequences():
    """2^21 sequences of 33 tokens of one channel: each is what it is in a batch of few (the same
    tiles and runs, so the same bits)."""
    B, T, D = 1 << 21, 33, 1
    x, dy = normal(B, T, D, seed=1), normal(B, T, D, seed=2)
    gate, h0 = normal(B, T, D, seed=3), normal(B, D, seed=4, dtype=F32)
    kw = dict(rate=torch.full((D,), 0.1, device=DEV), form="rate", scale="norm")
    dhT = normal(B, D, seed=5, dtype=F32)
    dx, dg, _, _, dh0 = gdn.glr_backward(dy, x, gate, h0, dhT, **kw)
    for at in (slice(0, 5), slice(B // 2 - 3, B // 2 + 3), slice(B - 5, B)):
        dx1, dg1, _, _, dh1 = gdn.glr_backward(dy[at], x[at], gate[at], h0[at], dhT[at], **kw)
        for a, b in ((dx, dx1), (dg, dg1), (dh0, dh1)):
            assert torch.equal(a[at], b)
    n = 5
    ref = L.glr(x[-n:].flatten(0, 1), gate[-n:].flatten(0, 1), None, kw["rate"], h0[-n:], [T] * n, "rate", "norm", dy[-n:].flatten(0, 1), dhT[-n:])
    for v, name in ((dx[-n:].flatten(0, 1), "dx"), (dg[-n:].flatten(0, 1), "dgate"), (dh0[-n:], "dh0")):
        close(v, ref[name], ref[name + "_err"] + ref[name].abs() * HALF[v.dtype] + 2.0 ** -120, name)


def test_very_many_short_prompts():
    """2^23 prompts of two tokens, a wave each: each is what it is among few (the same runs, so the
    same bits), and the recurrence in 64 bits."""
    B, T, D = 1 << 23, 2, 3
    x, gate, h0 = normal(B, T, D, seed=1), normal(B, T, D, seed=3), normal(B, D, seed=4, dtype=F32)
    kw = dict(form="sigmoid", scale="complement")
    y, hT = gdn.glr_forward(x, gate, h0, **kw)
    n = 5
    for at in (slice(0, n), slice(B // 2 - n, B // 2), slice(B - n, B)):
        y1, h1 = gdn.glr_forward(x[at], gate[at], h0[at], **kw)
        assert torch.equal(y[at], y1) and torch.equal(hT[at], h1)
        ref = L.glr(x[at].flatten(0, 1), gate[at].flatten(0, 1), None, None, h0[at], [T] * n, "sigmoid", "complement")
        close(y1.flatten(0, 1), ref["y"], ref["y_err"] + ref["y"].abs() * HALF[BF] + 2.0 ** -120, "y")
        close(h1, ref["hT"], ref["hT_err"] + ref["hT"].abs() * HALF[F32] + 2.0 ** -120, "hT")
