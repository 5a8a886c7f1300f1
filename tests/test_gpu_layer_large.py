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


def glr_last(x, gate, dy, kw, rows, lens, got, h0=None, dhT=None):
    """Results at the last rows [rows) of the last batch, in the first and the last channels, against
    the recurrence over those rows."""
    D = x.shape[-1]
    at = [0, 1, 63, D - 65, D - 2, D - 1]
    cut = lambda t: None if t is None else t[-1, rows][:, at]  # noqa: E731
    ref = L.glr(cut(x), cut(gate), None, kw["rate"][at], h0, lens, kw["form"], kw["scale"], cut(dy), dhT)
    y, hT, dx, dg, dh0 = got
    for v, name in ((cut(y), "y"), (cut(dx), "dx"), (cut(dg), "dgate"), (hT[-1:, at], "hT"), (None if dh0 is None else dh0[-1:, at], "dh0")):
        if v is not None:
            r = ref[name]
            close(v, r, ref[name + "_err"] + r.abs() * HALF[v.dtype] + 2.0 ** -120, name)


def test_glr_rows_past_2_to_the_31():
    """x, the gate, dy and what is written have 3.3e9 elements (6.7e9 bytes) each; the last batch begins
    past 2^31 elements and 2^32 bytes of every one."""
    B, T, D = 3, 8500, 1 << 17
    assert 2 * T * D > 1 << 31 and 2 * T * D * 2 > 1 << 32
    x, gate, dy = (normal(B, T, D, seed=i) for i in range(3))
    kw = dict(rate=torch.linspace(0.01, 0.2, D, device=DEV), form="rate", scale="norm")
    y, hT = gdn.glr_forward(x, gate, **kw)
    dx, dg, _, _, _ = gdn.glr_backward(dy, x, gate, **kw)
    glr_last(x, gate, dy, kw, slice(0, T), [T], (y, hT, dx, dg, None))


def test_glr_packed_rows_past_2_to_the_31():
    """One batch of packed sequences, the last of which begins past 2^31 elements and 2^32 bytes."""
    T, D, first = 17700, 1 << 17, 16500
    assert first * D > 1 << 31
    x, gate, dy = (normal(1, T, D, seed=i) for i in range(3))
    h0, dhT = normal(2, D, seed=4, dtype=F32), normal(2, D, seed=5, dtype=F32)
    cu = torch.tensor([0, first, T], dtype=torch.int32, device=DEV)
    kw = dict(rate=torch.linspace(0.01, 0.2, D, device=DEV), form="rate", scale="norm")
    y, hT = gdn.glr_forward(x, gate, h0, cu_seqlens=cu, **kw)
    dx, dg, _, _, dh0 = gdn.glr_backward(dy, x, gate, h0, dhT, cu_seqlens=cu, **kw)
    at = [0, 1, 63, D - 65, D - 2, D - 1]
    glr_last(x, gate, dy, kw, slice(first, T), [T - first], (y, hT, dx, dg, dh0), h0[1:, at], dhT[1:, at])


def test_layer_norm_rows_past_2_to_the_31():
    """Rows at a stride, a residual, both outputs; the last rows lie past 2^31 elements and 2^32 bytes."""
    rows, D, pad = (1 << 17) + 100, 16384, 8
    assert (rows - 4) * D > 1 << 31
    x = normal(rows, D + pad, seed=1)[:, :D]
    res, w, b = normal(rows, D, seed=2), normal(D, seed=3), normal(D, seed=4)
    last = slice(rows - 4, rows)
    y, s, _ = gdn.layer_norm_forward(x, w, b, res)
    ref, kept, h = L.layer_norm(x[last], w, b, res[last], 1e-5, BF)
    wd = w.cpu().double().abs()
    assert torch.equal(s[last].cpu().double(), kept)
    close(y[last], ref, ref.abs() * HALF[BF] + ((h.abs() + 1) * wd + b.cpu().double().abs()) * ARITH, "y")
    dy = x.contiguous()
    ds, _, _, _ = gdn.layer_norm_backward(dy, s, w, b, res)
    want, _, _ = L.layer_norm_grad(dy[last], kept, w, res[last], 1e-5)
    v = kept - kept.mean(-1, keepdim=True)
    r = (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    u, hs = dy[last].cpu().double().abs() * wd, h.abs() + 1
    size = res[last].cpu().double().abs() + r * (u + u.mean(-1, keepdim=True) + hs * (u * hs).mean(-1, keepdim=True))
    close(ds[last], want, want.abs() * HALF[BF] + size * ARITH, "ds")


def test_gate_norm_rows_past_2_to_the_31():
    """x by heads, the gate a part of wider rows; the last token of every tensor lies past 2^31
    elements and 2^32 bytes, or the last head does."""
    T, H, D = 4200, 64, 8192
    assert (T - 4) * H * D > 1 << 31 and (H - 1) * T * D > 1 << 31
    x = normal(H, T, D, seed=1).transpose(0, 1)
    z = normal(T, (H + 1) * D, seed=2)[:, D:].unflatten(-1, (H, D))
    w, dy = normal(H, D, seed=3), normal(T, H, D, seed=4)
    y = gdn.gate_norm_forward(x, z, w)
    dx, dz, _, _ = gdn.gate_norm_backward(dy, x, z, w)
    for t, h in ((slice(T - 2, T), slice(0, 2)), (slice(T - 2, T), slice(H - 2, H)), (slice(0, 2), slice(H - 2, H))):
        ref = L.gate_norm(x[t, h], z[t, h], w[h], None, 1e-5, "silu", False, False, dy[t, h])
        for v, name in ((y, "y"), (dx, "dx"), (dz, "dz")):
            close(v[t, h], ref[name], ref[name].abs() * HALF[BF] + ref[name + "size"] * ARITH, name)
