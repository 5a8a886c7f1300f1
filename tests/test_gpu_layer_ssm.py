"""Selective state space scan on the GPU against its recurrence in 64 bits.

Tolerances, from sums of the terms' sizes (the same recurrence with every factor
replaced by its size), Y for y, Z for the states:
  fp32 io: products and their sums in fp32.  A chunk adds 64 terms to a sum, a
    state goes through one product and at most 64 additions a chunk and fades
    with its decays; exponentials and softplus are good to a few units.  All in
    all at most 2^9 roundings of 2^-24: 2^-15 of the terms' size.
  bf16 io: y's operands are rounded once each, three of them on one way (the
    weighted value into the state, the state into y or the chunk's matrix into
    y): 2 * 2^-8 Y, and 2^-8 |y| for y itself.  The states that leave the
    kernel take weighted values of three bf16 parts, 2^-27: fp32's 2^-15 Z.
  dx as y (with its own sizes); dB, dC: the chunk's matrix once, 2^-8 of the
    terms, and 2^-8 of the result; ddt, dA: fp32 throughout, but for a gate the
    differences of up to four chunks' sums: 2^-15 of the sizes of all pairs
    that meet the 256 tokens around."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FP = 2.0 ** -15


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def close(got, ref, tol, what):
    d = (got.detach().cpu().double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e over its tolerance" % (what, int(bad.sum()), bad.numel(),
                                                                               float((d - tol).max()))


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(DEV)


def inputs(B, T, H, P, N, G, dt, dtt, n, h0, seed=0, strong=False, joint=True):
    """x, B and C side by side in one buffer, as a convolution leaves them."""
    buf = rnd(B, T, H * P + 2 * G * N, seed=seed + 1, dtype=dt)
    x, Bm, Cm = buf.split((H * P, G * N, G * N), -1)
    d = dict(x=x.unflatten(-1, (H, P)), B=Bm.unflatten(-1, (G, N)), C=Cm.unflatten(-1, (G, N)))
    if not joint:
        d = {k: v.contiguous() for k, v in d.items()}
    wide = rnd(B, T, H + 3, seed=seed + 2, dtype=dtt)
    d["dt"] = wide[..., 2:2 + H]
    g = torch.Generator().manual_seed(seed + 3)
    lo, hi = (0.5, 3.0) if strong else (1e-3, 1e-1)
    dt0 = torch.exp(torch.rand(H, generator=g) * (torch.tensor(hi).log() - torch.tensor(lo).log()) + torch.tensor(lo).log())
    d["dt_bias"] = (dt0 + torch.log(-torch.expm1(-dt0))).to(DEV)
    d["A"] = (-(1 + 15 * torch.rand(H, generator=g))).to(DEV)
    d["D"] = rnd(H, seed=seed + 4)
    d["h0"] = rnd(n, H, N, P, seed=seed + 5) if h0 else None
    return d


def forward(d, **kw):
    return gdn.ssm_forward(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], d["h0"], **kw)


def flat(t):
    return t.reshape(-1, *t.shape[2:])


CASES = [  # lens (batch, tokens; or packed), H, P, N, G, type, dt's type, h0, softplus, strong gates
    ((1, 1), 2, 64, 64, 1, BF, BF, False, True, False), ((2, 63), 3, 64, 128, 1, BF, F32, True, True, False),
    ((1, 64), 4, 128, 64, 2, BF, BF, True, True, False), ((1, 65), 2, 128, 128, 2, F32, F32, True, True, False),
    ((1, 300), 2, 64, 64, 2, BF, BF, True, False, False), ((2, 700), 4, 64, 128, 2, BF, BF, True, True, False),
    ((1, 1100), 1, 128, 128, 1, BF, F32, False, True, False), ((1, 600), 3, 64, 64, 3, F32, F32, True, True, False),
    ((1, 520), 2, 128, 64, 1, F32, F32, False, True, False), ((1, 400), 4, 64, 128, 1, BF, BF, True, True, True),
    ([70, 0, 1, 256, 64, 0, 5], 4, 64, 128, 2, BF, BF, True, True, False),
    ([0, 0, 3], 2, 128, 128, 1, BF, BF, True, True, False), ([600, 30], 1, 64, 64, 1, BF, F32, False, True, False),
    ([1] * 70, 2, 64, 64, 1, F32, F32, True, True, False), ([257, 1, 300], 2, 128, 128, 2, BF, BF, True, True, True)]


@pytest.mark.parametrize("lens,H,P,N,G,dt,dtt,h0,softplus,strong", CASES)
def test_forward_and_backward(lens, H, P, N, G, dt, dtt, h0, softplus, strong):
    packed = isinstance(lens, list)
    B, T = (1, sum(lens)) if packed else lens
    each = lens if packed else [T] * B
    n = len(each)
    d = inputs(B, T, H, P, N, G, dt, dtt, n, h0, strong=strong)
    if not softplus:
        d["dt"], d["dt_bias"] = d["dt"].abs() * 0.1, None
    cu = offsets(lens) if packed else None
    y, hT = forward(d, dt_softplus=softplus, cu_seqlens=cu)
    step, raw = L.step_sizes(flat(d["dt"]), d["dt_bias"], softplus)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], each)
    ref, rT = L.ssm(*args)
    Y, Z = L.ssm(*args, absolute=True)
    b = dt is BF
    close(flat(y), ref, ref.abs() * HALF[dt] + Y * (2 * 2.0 ** -8 * b + FP), "y")
    close(hT, rT, Z * FP, "hT")
    # without a final state the segments' starts are rounded like y's other operands
    alone, none = forward(d, cu_seqlens=cu, dt_softplus=softplus, output_final_state=False)
    assert none is None
    close(flat(alone), ref, ref.abs() * HALF[dt] + Y * (2 * 2.0 ** -8 * b + FP), "y without a final state")

    dy, dhT = rnd(B, T, H, P, seed=8, dtype=dt), rnd(n, H, N, P, seed=9)
    got = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], d["h0"], dhT,
                           dt_softplus=softplus, cu_seqlens=cu)
    dx, ddt, dA, dB, dC, dD, dbias, dh0 = got
    g = L.ssm_grad(flat(dy), *args[:7], each, dhT)
    a = L.ssm_grad(flat(dy), *args[:7], each, dhT, absolute=True)
    close(flat(dx), g["dx"], g["dx"].abs() * HALF[dt] + a["dx"] * (2 * 2.0 ** -8 * b + FP), "dx")
    for k, v in (("dB", dB), ("dC", dC)):
        close(flat(v), g[k], g[k].abs() * HALF[dt] + a[k] * (2.0 ** -8 * b + FP), k)
    close(dD, g["dD"], (flat(dy).cpu().double() * flat(d["x"]).cpu().double()).abs().sum((0, 2)) * FP, "dD")
    # pairs that meet the 256 tokens on either side, sequence by sequence
    near, at = torch.zeros_like(a["pairs"]), 0
    for k in each:
        c = torch.cat([torch.zeros(1, H, dtype=torch.float64), a["pairs"][at:at + k].cumsum(0)])
        i = torch.arange(k)
        near[at:at + k] = c[(i + 257).clamp(max=k)] - c[(i - 256).clamp(min=0)]
        at += k
    slope = torch.sigmoid(raw) if softplus else 1.0
    size = (a["ddt"] + near * d["A"].cpu().double().abs()) * slope
    want = g["ddt"] * slope
    close(flat(ddt), want, want.abs() * HALF[dtt] + size * FP, "ddt")
    close(dA, g["dA"], (near * step).sum(0) * FP, "dA")
    if dbias is not None:
        close(dbias, want.sum(0), size.sum(0) * FP, "ddt_bias")
    else:
        assert d["dt_bias"] is None
    if dh0 is not None:
        close(dh0, g["dh0"], a["dh0"] * FP, "dh0")
    else:
        assert d["h0"] is None


def test_gradients_without_a_final_states_gradient():
    d = inputs(1, 900, 2, 64, 64, 1, BF, BF, 1, True)
    dy = rnd(1, 900, 2, 64, seed=8, dtype=BF)
    a = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], d["h0"])
    b = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], d["h0"], torch.zeros_like(d["h0"]))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    c = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"])
    assert c[5] is None and c[6] is None and c[7] is None


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("P,N", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_steps_are_the_recurrence(P, N, dt):
    """Steps in fp32 from a pool of states; a product, a sum and two
    exponentials a step: 2^-20 of the terms' size after ten of them."""
    B, T, H, G = 3, 10, 4, 2
    d = inputs(B, T, H, P, N, G, dt, dt, B, True)
    step, _ = L.step_sizes(flat(d["dt"]), d["dt_bias"], True)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [T] * B)
    ref, rT = L.ssm(*args)
    Y, Z = L.ssm(*args, absolute=True)
    pool = torch.full((5, H, N, P), float("nan"), device=DEV)
    slots = torch.tensor([3, 0, 4], device=DEV, dtype=torch.int32)
    pool[slots.long()] = d["h0"]
    ys = [gdn.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], pool, d["D"], d["dt_bias"], slots=slots)
          for t in range(T)]
    y = torch.stack(ys, 1)
    close(flat(y), ref, ref.abs() * HALF[dt] + Y * 2.0 ** -18, "y")
    close(pool[slots.long()], rT, Z * 2.0 ** -20, "state")
    assert pool[[1, 2]].isnan().all()
    direct = d["h0"].clone()
    for t in range(T):
        one = gdn.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], direct, d["D"], d["dt_bias"])
        assert torch.equal(one, ys[t])


def test_step_padding_and_repeated_slots():
    B, H, P, N = 70, 2, 64, 64
    d = inputs(B, 1, H, P, N, 1, BF, BF, 1, False)
    one = {k: d[k][:, 0] for k in ("x", "dt", "B", "C")}
    pool = rnd(80, H, N, P, seed=3)
    slots = torch.randperm(80, generator=torch.Generator().manual_seed(4))[:B].to(torch.int32).to(DEV)
    slots[5], slots[6], slots[7] = -1, 80, -2 ** 31
    slots[66] = slots[2]
    slots[67] = slots[2]
    before = pool.clone()
    y = gdn.ssm_step(one["x"], one["dt"], d["A"], one["B"], one["C"], pool, d["D"], d["dt_bias"], slots=slots)
    pad = [5, 6, 7, 66, 67]
    keep = [i for i in range(B) if i not in pad]
    alone = before.clone()
    ref = gdn.ssm_step(one["x"][keep], one["dt"][keep], d["A"], one["B"][keep], one["C"][keep], alone, d["D"], d["dt_bias"],
                       slots=slots[keep])
    assert y[pad].eq(0).all() and torch.equal(y[keep], ref) and torch.equal(pool, alone)
    assert gdn.ssm_step(one["x"][:0], one["dt"][:0], d["A"], one["B"][:0], one["C"][:0], pool).shape == (0, H, P)


def test_segments_and_single_pass_agree():
    """A long stream alone is cut into segments; the same tokens as two calls, the
    second from the first one's state, give the same numbers."""
    d = inputs(1, 2000, 4, 64, 128, 2, BF, BF, 1, True)
    y, hT = forward(d)
    cut = 256
    parts = [{k: (v[:, s] if k in ("x", "dt", "B", "C") else v) for k, v in d.items()} for s in (slice(0, cut), slice(cut, 2000))]
    y0, h1 = forward(parts[0])
    parts[1]["h0"] = h1
    y1, h2 = forward(parts[1])
    step, _ = L.step_sizes(flat(d["dt"]), d["dt_bias"], True)
    Y, Z = L.ssm(flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [2000], absolute=True)
    both = torch.cat([y0, y1], 1)
    # each way within y's tolerance of the recurrence
    close(flat(y), flat(both).cpu().double(), 2 * (flat(both).cpu().double().abs() * 2.0 ** -8 + Y * (2 * 2.0 ** -8 + FP)), "y")
    close(hT, h2.cpu().double(), Z * 2 * FP, "hT")


def test_gates_at_their_ends():
    """A = 0 (nothing fades), dt = 0 (a token without effect) and gates so strong
    that every decay is 0: finite, and what the recurrence gives."""
    T, H, P, N = 200, 3, 64, 64
    d = inputs(1, T, H, P, N, 1, BF, F32, 1, True)
    d["A"] = torch.tensor([0.0, -1.0, -1e4], device=DEV)
    d["dt"] = rnd(1, T, H, seed=5).abs() * 0.05
    d["dt"][:, ::3] = 0.0
    d["dt_bias"] = None
    y, hT = forward(d, dt_softplus=False)
    step, _ = L.step_sizes(flat(d["dt"]), None, False)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [T])
    ref, rT = L.ssm(*args)
    Y, Z = L.ssm(*args, absolute=True)
    close(flat(y), ref, ref.abs() * 2.0 ** -8 + Y * (2 * 2.0 ** -8 + FP), "y")
    close(hT, rT, Z * FP, "hT")
    dy = rnd(1, T, H, P, seed=8, dtype=BF)
    got = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], None, d["h0"], dt_softplus=False)
    assert all(t.isfinite().all() for t in got if t is not None)


def test_weak_gates_behind_strong_ones():
    """A decay of e^-2000 early in each chunk and gates of 1e-5 behind it: a sum of
    gates held in 32 bits would be off by 2^-14 there, all later decays with it."""
    T, H, P, N = 128, 1, 64, 64
    d = inputs(1, T, H, P, N, 1, F32, F32, 1, False)
    d["A"], d["dt_bias"], d["D"] = torch.tensor([-1.0], device=DEV), None, None
    d["dt"] = torch.full((1, T, H), 1e-5, device=DEV)
    d["dt"][:, 1] = 2000.0
    d["dt"][:, 65] = 2000.0
    y, hT = forward(d, dt_softplus=False)
    step, _ = L.step_sizes(flat(d["dt"]), None, False)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), None, None, [T])
    ref, rT = L.ssm(*args)
    Y, Z = L.ssm(*args, absolute=True)
    close(flat(y), ref, Y * 2.0 ** -18, "y")
    close(hT, rT, Z * 2.0 ** -18, "hT")


def test_a_gate_that_clears_the_state():
    """A token whose decay is e^-1e20 clears the state; the decays of the tokens
    behind it are those without it."""
    T, H, P, N = 150, 1, 64, 64
    d = inputs(1, T, H, P, N, 1, F32, F32, 1, True)
    d["A"], d["dt_bias"], d["D"] = torch.tensor([-1.0], device=DEV), None, None
    d["dt"] = rnd(1, T, H, seed=5).abs() * 0.02
    at = 70
    alone = {k: (v[:, at + 1:] if k in ("x", "dt", "B", "C") else v) for k, v in d.items()}
    alone["x"], alone["h0"] = alone["x"].contiguous(), None
    d["dt"][:, at] = 1e20
    d["x"] = d["x"].clone()
    d["x"][:, at] = 0.0
    y, hT = forward(d, dt_softplus=False)
    ref, rT = forward(alone, dt_softplus=False)
    step, _ = L.step_sizes(flat(alone["dt"]), None, False)
    Y, Z = L.ssm(flat(alone["x"]), step, d["A"], flat(alone["B"]), flat(alone["C"]), None, None, [T - at - 1], absolute=True)
    close(flat(y[:, at + 1:]), flat(ref).double().cpu(), Y * 2.0 ** -15, "y")
    close(hT, rT.double().cpu(), Z * 2.0 ** -15, "hT")


@pytest.mark.parametrize("name", ["x", "B", "C", "dt"])
def test_a_nan_reaches_its_chunk_and_what_follows(name):
    """...and neither the chunks before it nor another sequence."""
    lens, H, P, N = [150, 90], 2, 64, 64
    d = inputs(1, 240, H, P, N, 1, BF, BF, 2, True)
    cu = offsets(lens)
    dy = rnd(1, 240, H, P, seed=8, dtype=BF)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    y, hT = forward(d, cu_seqlens=cu)
    g = gdn.ssm_backward(dy, *(d[k] for k in names), cu_seqlens=cu)
    d[name] = d[name].clone() if name in ("x", "dt") else d[name]
    d[name][:, 70] = float("nan")
    z, kT = forward(d, cu_seqlens=cu)
    h = gdn.ssm_backward(dy, *(d[k] for k in names), cu_seqlens=cu)
    assert torch.equal(z[:, :64], y[:, :64]) and torch.equal(z[:, 150:], y[:, 150:]) and torch.equal(kT[1], hT[1])
    assert z[:, 70].isnan().any()
    for k in (0, 1, 3, 4):
        assert torch.equal(h[k][:, 150:], g[k][:, 150:])
    assert torch.equal(h[7][1], g[7][1])


def test_rows_behind_the_sequences_and_malformed_offsets():
    lens, T, H, P, N = [30, 0, 100], 160, 2, 64, 64
    d = inputs(1, T, H, P, N, 1, BF, BF, 3, True)
    for k in ("x", "B", "C", "dt"):
        d[k][:, 130:] = float("nan")
    cu = offsets(lens)
    y = torch.full((1, T, H, P), 7.0, device=DEV, dtype=BF)
    _, hT = forward(d, cu_seqlens=cu, y=y)
    cutd = {k: (v[:, :130] if k in ("x", "dt", "B", "C") else v) for k, v in d.items()}
    ref, rT = forward(cutd, cu_seqlens=cu)
    assert torch.equal(y[:, :130], ref) and y[:, 130:].eq(7.0).all() and torch.equal(hT, rT) and hT.isfinite().all()
    assert torch.equal(hT[1], d["h0"][1])                        # an empty sequence keeps its state
    dy = rnd(1, T, H, P, seed=8, dtype=BF)
    dy[:, 130:] = float("nan")
    grads = {k: torch.full_like(d[k].contiguous(), 7.0) for k in ("x", "B", "C", "dt")}
    one = torch.full((1, T, H * P + 2 * N), 7.0, device=DEV, dtype=BF)
    dx, dB, dC = one.split((H * P, N, N), -1)
    out = dict(dx=dx.unflatten(-1, (H, P)), dB=dB.unflatten(-1, (1, N)), dC=dC.unflatten(-1, (1, N)), ddt=grads["dt"])
    a = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], d["h0"], cu_seqlens=cu, **out)
    b = gdn.ssm_backward(dy[:, :130].contiguous(), *(cutd[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")), cu_seqlens=cu)
    for u, v in zip(a, b):
        same = u[:, :130] if u.dim() > 1 and u.shape[:2] == (1, T) else u
        assert torch.equal(same, v) and v.isfinite().all()
    assert one[:, 130:].eq(7.0).all() and grads["dt"][:, 130:].eq(7.0).all()
    # (the last two: more segments than a list in order can have)
    for bad, T in (([0, 1000, 160], T), ([-5, 60, 20, 160], T), ([150, 10], T), ([2 ** 31 - 1, -2 ** 31], T),
                   ([0, 1100, 0, 1100], 1100), ([0, 3000, 0, 3000, 0, 3000, 0, 3000], 3000)):
        m = inputs(1, T, H, P, N, 1, BF, BF, len(bad) - 1, True)
        off = torch.tensor(bad, device=DEV, dtype=torch.int32)
        forward(m, cu_seqlens=off)
        gdn.ssm_backward(rnd(1, T, H, P, seed=8, dtype=BF), *(m[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")), cu_seqlens=off)
    torch.cuda.synchronize()


def test_dense_and_side_by_side_inputs_agree():
    a, b = (inputs(2, 130, 4, 64, 64, 2, BF, BF, 2, True, joint=j) for j in (True, False))
    ya, ha = forward(a)
    yb, hb = forward(b)
    assert torch.equal(ya, yb) and torch.equal(ha, hb)


def test_empty_and_refused():
    d = inputs(2, 10, 2, 64, 64, 1, F32, F32, 2, True)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    none = {k: (v[:, :0] if k in ("x", "dt", "B", "C") else v) for k, v in d.items()}
    y, hT = forward(none)
    assert y.shape == (2, 0, 2, 64) and torch.equal(hT, d["h0"])
    g = gdn.ssm_backward(y, *(none[k] for k in names), d["h0"])
    assert g[2].eq(0).all() and g[5].eq(0).all() and g[6].eq(0).all() and torch.equal(g[7], d["h0"])
    f = lambda **kw: gdn.ssm_forward(*({**d, **kw}[k] for k in names))  # noqa: E731
    for bad, err in ((lambda: f(x=d["x"].to(BF)), TypeError), (lambda: f(A=d["A"][:1]), ValueError),
                     (lambda: f(dt=d["dt"].double()), TypeError), (lambda: f(h0=d["h0"][:1]), ValueError),
                     (lambda: f(C=d["C"].contiguous()), ValueError), (lambda: f(D=d["D"].to(BF)), TypeError),
                     (lambda: f(x=d["x"][..., :32].contiguous(), h0=None), gdn.GdnError),
                     (lambda: f(x=d["x"][:, :1].expand(2, 10, 2, 64)), gdn.GdnError),
                     (lambda: gdn.ssm_forward(*(d[k] for k in names), hT=d["h0"]), ValueError),
                     (lambda: gdn.ssm_forward(*(d[k] for k in names), cu_seqlens=offsets([20])), ValueError),
                     (lambda: gdn.ssm_forward(*(d[k] for k in names), stream=torch.cuda.Stream(), y=d["x"]), ValueError)):
        with pytest.raises(err):
            bad()


def test_gradient_against_differences():
    """fp32 io: a difference over 2 h, h = 2^-8, of a loss known to 2^-15 of its
    terms, so to 2^-8 of them over h; and a third derivative of the same sizes."""
    H, P, N, h = 2, 64, 64, 2.0 ** -8
    d = inputs(1, 300, H, P, N, 1, F32, F32, 1, True, joint=False)
    d["dt"] = d["dt"].contiguous()
    dy, dhT = rnd(1, 300, H, P, seed=8), rnd(1, H, N, P, seed=9, scale=0.1)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")

    def loss(v):
        y, hT = gdn.ssm_forward(*v)
        return float((y.double() * dy.double()).sum() + (hT.double() * dhT.double()).sum())

    leaves = [d[k] for k in names]
    g = gdn.ssm_backward(dy, *leaves, dhT)
    step, _ = L.step_sizes(flat(d["dt"]), d["dt_bias"], True)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [300])
    Y, Z = L.ssm(*args, absolute=True)
    terms = float((Y * dy[0].cpu().double().abs()).sum() + (Z * dhT.cpu().double().abs()).sum())
    for i, name in enumerate(names):
        v = rnd(*leaves[i].shape, seed=20 + i)
        plus, minus = list(leaves), list(leaves)
        plus[i], minus[i] = leaves[i] + h * v, leaves[i] - h * v
        num = (loss(plus) - loss(minus)) / (2 * h)
        assert abs(num - float((g[i].double() * v.double()).sum())) <= terms * 2.0 ** -7, name


def test_streams_graphs_and_repeats():
    d = inputs(2, 700, 4, 64, 128, 2, BF, BF, 2, True)
    dy = rnd(2, 700, 4, 64, seed=8, dtype=BF)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    pool0 = rnd(3, 4, 128, 64, seed=9)
    pool = pool0.clone()
    slots = torch.tensor([2, 0], device=DEV, dtype=torch.int32)

    def work():
        pool.copy_(pool0)
        y, hT = forward(d)
        s = gdn.ssm_step(d["x"][:, 5], d["dt"][:, 5], d["A"], d["B"][:, 5], d["C"][:, 5], pool, d["D"], d["dt_bias"], slots=slots)
        return [y, hT, s, *gdn.ssm_backward(dy, *(d[k] for k in names))]

    ref = [t.clone() for t in work()]
    assert all(torch.equal(a, b) for a, b in zip(ref, work()))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, hT = forward(d, stream=st)
    st.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(hT, ref[1])
    # two at once, each with its own workspace
    st2 = torch.cuda.Stream()
    a = [forward(d, stream=s) for s in (st, st2, st, st2)]
    torch.cuda.synchronize()
    assert all(torch.equal(u[0], ref[0]) and torch.equal(u[1], ref[1]) for u in a)
    with torch.cuda.stream(st):
        work()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        d["x"].copy_(rnd(2, 700, 4, 64, seed=10 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, work())), k


def test_given_workspace_and_outputs():
    d = inputs(1, 1500, 2, 64, 64, 1, BF, BF, 1, True)
    y, hT = forward(d)
    y2, h2 = torch.empty_like(y), torch.empty_like(hT)
    ws = torch.full((1 << 22,), 0xff, device=DEV, dtype=torch.uint8)      # NaN in every type
    got = forward(d, y=y2, hT=h2, workspace=ws)
    assert got[0] is y2 and got[1] is h2 and torch.equal(y, y2) and torch.equal(hT, h2)
    with pytest.raises(gdn.GdnError) as e:
        forward(d, workspace=ws[:1024])
    assert e.value.status == 6
    dy = rnd(1, 1500, 2, 64, seed=8, dtype=BF)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    a = gdn.ssm_backward(dy, *(d[k] for k in names))
    b = gdn.ssm_backward(dy, *(d[k] for k in names), workspace=torch.full((1 << 25,), 0xff, device=DEV, dtype=torch.uint8))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_gradients_that_overlap_are_refused():
    b, T, H, P, N, G = 2, 70, 2, 64, 64, 1
    d = inputs(b, T, H, P, N, G, BF, BF, 1, False)
    dy = rnd(b, T, H, P, seed=8, dtype=BF)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    run = lambda *g: gdn.ssm_backward(dy, *(d[k] for k in names), dx=g[0], dB=g[1], dC=g[2])  # noqa: E731
    new = lambda w: torch.empty(b, T, w, device=DEV, dtype=BF)  # noqa: E731
    part = lambda t, at, heads, n: t[..., at:at + heads * n].unflatten(-1, (heads, n))  # noqa: E731
    ref = gdn.ssm_backward(dy, *(d[k] for k in names))
    both = new(256)
    got = run(part(both, 0, H, P), part(both, 128, G, N), part(both, 192, G, N))
    wide = [new(256) for _ in range(3)]                      # or three buffers
    also = run(*(part(t, 0, h, 64) for t, h in zip(wide, (H, G, G))))
    for k in (0, 3, 4):
        assert torch.equal(got[k], ref[k]) and torch.equal(also[k], ref[k])
    for at in ((0, 64, 192), (0, 128, 128), (64, 128, 0), (0, 128, 160)):
        with pytest.raises(ValueError):
            run(part(both, at[0], H, P), part(both, at[1], G, N), part(both, at[2], G, N))
    with pytest.raises(ValueError):
        run(part(wide[0], 0, H, P), part(wide[1], 0, G, N), part(wide[1], 64 - 8, G, N))


def test_tokens_behind_32_bit_offsets():
    """More than 2^32 bytes of x: the last tokens are those of a run of their own from
    the state before them.  Either is off by at most 2 2^-8 of the terms' sizes and a
    rounding (see above), of which 2^-6 of the result's norm leaves room for both."""
    T, H, P, N, k = (1 << 17) + 77, 128, 128, 64, 700
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s, dtype=BF: torch.randn(*s, generator=g, device=DEV, dtype=dtype)  # noqa: E731
    x, dy, B, C = new(1, T, H, P), new(1, T, H, P), new(1, T, 1, N), new(1, T, 1, N)
    dt, A = new(1, T, H, dtype=F32), -torch.rand(H, generator=g, device=DEV) - 0.1
    assert x.numel() * 2 > 1 << 32
    rest = dict(D=new(H, dtype=F32), dt_bias=torch.full((H,), -3.0, device=DEV))
    y, hT = gdn.ssm_forward(x, dt, A, B, C, **rest)
    grads = gdn.ssm_backward(dy, x, dt, A, B, C, **rest)
    _, before = gdn.ssm_forward(x[:, :T - k], dt[:, :T - k], A, B[:, :T - k], C[:, :T - k], **rest)
    tail = [t[:, T - k:] for t in (x, dt, B, C)]
    y2, h2 = gdn.ssm_forward(tail[0], tail[1], A, *tail[2:], **rest, h0=before)
    grads2 = gdn.ssm_backward(dy[:, T - k:], tail[0], tail[1], A, *tail[2:], **rest, h0=before)
    off = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    assert off(y[:, T - k:], y2) < 2.0 ** -6 and off(hT, h2) < 2.0 ** -12
    for i in (0, 1, 3, 4):
        assert off(grads[i][:, T - k:], grads2[i]) < 2.0 ** -6, i


def test_slots_behind_32_bit_offsets():
    S, H, P, N = 1100, 64, 128, 128
    pool = torch.zeros(S, H, N, P, device=DEV)
    assert pool.numel() * 4 > 1 << 32
    d = inputs(3, 1, H, P, N, 8, BF, BF, 3, True)
    one = {k: d[k][:, 0] for k in ("x", "dt", "B", "C")}
    slots = torch.tensor([S - 1, 5, 1024], device=DEV, dtype=torch.int32)
    pool[slots.long()] = d["h0"]
    small = d["h0"].clone()
    args = (one["x"], one["dt"], d["A"], one["B"], one["C"])
    y = gdn.ssm_step(*args, pool, d["D"], d["dt_bias"], slots=slots)
    ref = gdn.ssm_step(*args, small, d["D"], d["dt_bias"])
    assert torch.equal(y, ref) and torch.equal(pool[slots.long()], small)


@pytest.mark.parametrize("H,P,N,G,dt", [(4, 64, 64, 1, BF), (2, 128, 64, 2, F32)])
def test_gradients_of_single_tokens_in_a_batch(H, P, N, G, dt):
    """T = 1 and several batches: parts of one buffer, which hold what the binding's
    own outputs do, with nothing written beside them; tensors of their own have no
    common stride between batches and are refused."""
    b = 3
    d = inputs(b, 1, H, P, N, G, dt, dt, b, True)
    dy = rnd(b, 1, H, P, seed=8, dtype=dt)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    ref = gdn.ssm_backward(dy, *(d[k] for k in names))
    step, raw = L.step_sizes(flat(d["dt"]), d["dt_bias"], True)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [1] * b)
    g, a = (L.ssm_grad(flat(dy), *args, None, absolute=k) for k in (False, True))
    for k, v in (("dx", ref[0]), ("dB", ref[3]), ("dC", ref[4])):
        close(flat(v), g[k], g[k].abs() * HALF[dt] + a[k] * (2 * 2.0 ** -8 * (dt is BF) + FP), k)
    wide = torch.full((b, 1, H * P + 2 * G * N + 64), 7.0, device=DEV, dtype=dt)
    dx, dB, dC, rest = wide.split((H * P, G * N, G * N, 64), -1)
    one = dict(dx=dx.unflatten(-1, (H, P)), dB=dB.unflatten(-1, (G, N)), dC=dC.unflatten(-1, (G, N)))
    got = gdn.ssm_backward(dy, *(d[k] for k in names), **one)
    assert all(torch.equal(u, v) for u, v in zip(got, ref)) and rest.eq(7.0).all()
    with pytest.raises(ValueError, match="same strides"):
        gdn.ssm_backward(dy, *(d[k] for k in names), dx=torch.empty_like(dy), dB=torch.empty(b, 1, G, N, device=DEV, dtype=dt),
                         dC=torch.empty(b, 1, G, N, device=DEV, dtype=dt))


@pytest.mark.parametrize("lens,H,P,N,G,dt", [
    ((1, 2000), 4, 64, 128, 2, BF), ((2, 100), 2, 128, 128, 1, BF), ((1, 1500), 1, 128, 64, 1, BF),
    ([70, 0, 600, 1, 256], 4, 64, 64, 2, BF), ([1000, 30], 3, 64, 128, 3, BF), ((1, 700), 2, 64, 64, 1, F32)])
def test_the_final_state_changes_nothing_else(lens, H, P, N, G, dt):
    """y has the same bits whether or not the final state is asked for, for
    sequences of one segment and of several."""
    packed = isinstance(lens, list)
    B, T = (1, sum(lens)) if packed else lens
    n = len(lens) if packed else B
    d = inputs(B, T, H, P, N, G, dt, dt, n, True)
    cu = offsets(lens) if packed else None
    y, hT = forward(d, cu_seqlens=cu)
    alone, none = forward(d, cu_seqlens=cu, output_final_state=False)
    assert none is None and hT is not None and torch.equal(y, alone)


@pytest.mark.parametrize("H,P,N,G,dt", [(4, 64, 128, 2, BF), (2, 128, 64, 1, BF), (2, 64, 64, 2, F32)])
def test_many_packed_sequences_are_each_their_own(H, P, N, G, dt):
    """Two hundred short sequences and a few long ones between them: every one has the
    bits of a call of its own (the long ones within rounding: their segments differ)."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 90, (200,), generator=g).tolist()
    lens[20], lens[77], lens[140], lens[199] = 700, 64, 0, 1300
    n, T = len(lens), sum(lens)
    d = inputs(1, T, H, P, N, G, dt, F32, n, True)
    cu = offsets(lens)
    dy, dhT = rnd(1, T, H, P, seed=8, dtype=dt), rnd(n, H, N, P, seed=9)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    y, hT = forward(d, cu_seqlens=cu)
    grads = gdn.ssm_backward(dy, *(d[k] for k in names), dhT, cu_seqlens=cu)
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    for k in [0, 1, 19, 20, 21, 76, 77, 78, 140, 141, 198, 199]:
        s = slice(at[k], at[k + 1])
        one = {m: (v[:, s] if m in ("x", "dt", "B", "C") else v[k:k + 1] if m == "h0" else v) for m, v in d.items()}
        y1, h1 = forward(one)
        g1 = gdn.ssm_backward(dy[:, s].contiguous(), *(one[m] for m in names), dhT[k:k + 1])
        pairs = [(y[:, s], y1), (hT[k:k + 1], h1), (grads[7][k:k + 1], g1[7])] + [(grads[i][:, s], g1[i]) for i in (0, 1, 3, 4)]
        for u, v in pairs:
            if lens[k] < 256:
                assert torch.equal(u, v), k
            else:
                assert float((u.double() - v.double()).norm()) <= 2.0 ** -6 * float(v.double().norm()), k


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("lens", [(2, 150), [100, 0, 64, 37], (1, 700)])
def test_a_gate_of_minus_infinity(lens, dt):
    """A = -inf: every token clears the state before it, also where a sequence ends
    inside a chunk.  (dt's gradient has A times a zero there: no number.)"""
    packed = isinstance(lens, list)
    B, T = (1, sum(lens)) if packed else lens
    each = lens if packed else [T] * B
    n, H, P, N = len(each), 2, 64, 64
    d = inputs(B, T, H, P, N, 1, dt, F32, n, True)
    d["A"] = torch.tensor([float("-inf"), -2.0], device=DEV)
    d["dt"], d["dt_bias"] = rnd(B, T, H, seed=5).abs() * 0.1 + 0.01, None
    cu = offsets(lens) if packed else None
    y, hT = forward(d, dt_softplus=False, cu_seqlens=cu)
    args = (flat(d["x"]), flat(d["dt"]), d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], each)
    ref, rT = L.ssm(*args)
    Y, Z = L.ssm(*args, absolute=True)
    b = dt is BF
    close(flat(y), ref, ref.abs() * HALF[dt] + Y * (2 * 2.0 ** -8 * b + FP), "y")
    close(hT, rT, Z * FP, "hT")
    dy, dhT = rnd(B, T, H, P, seed=8, dtype=dt), rnd(n, H, N, P, seed=9)
    dx, ddt, dA, dB, dC, dD, _, dh0 = gdn.ssm_backward(dy, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], None, d["h0"], dhT,
                                                       dt_softplus=False, cu_seqlens=cu)
    g = L.ssm_grad(flat(dy), *args, dhT)
    a = L.ssm_grad(flat(dy), *args, dhT, absolute=True)
    close(flat(dx), g["dx"], g["dx"].abs() * HALF[dt] + a["dx"] * (2 * 2.0 ** -8 * b + FP), "dx")
    for k, v in (("dB", dB), ("dC", dC)):
        close(flat(v), g[k], g[k].abs() * HALF[dt] + a[k] * (2.0 ** -8 * b + FP), k)
    close(dh0, g["dh0"], a["dh0"] * FP, "dh0")
    close(dA, g["dA"], (a["pairs"] * flat(d["dt"]).cpu().double()).sum(0) * FP, "dA")
    assert ddt[..., 1].isfinite().all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("P,N,dt", [(64, 128, BF), (128, 64, BF), (128, 128, F32), (64, 64, F32)])
def test_tokens_before_a_nan_do_not_see_it(name, value, P, N, dt):
    """A token's y is of the tokens up to it: NaN and infinity behind it, in its chunk
    or later, leave it as it is, as single-token steps do."""
    B, T, H, G, bad = 2, 150, 4, 2, 101
    d = inputs(B, T, H, P, N, G, dt, dt, B, True)
    step, _ = L.step_sizes(flat(d["dt"]), d["dt_bias"], True)
    args = (flat(d["x"]), step, d["A"], flat(d["B"]), flat(d["C"]), d["D"], d["h0"], [T] * B)
    ref, _ = L.ssm(*args)
    Y, _ = L.ssm(*args, absolute=True)
    clean, hT = forward(d)
    d[name][0, bad] = value
    y, kT = forward(d)
    tol = ref.abs() * HALF[dt] + Y * (2 * 2.0 ** -8 * (dt is BF) + FP)
    before = slice(0, bad)                              # of the first batch
    close(flat(y)[before], ref[before], tol[before], "y before")
    assert torch.equal(y[1], clean[1]) and torch.equal(kT[1], hT[1])
    if name == "C":                                     # only its own token reads C
        close(flat(y)[bad + 1:], ref[bad + 1:], tol[bad + 1:], "y behind")
        assert torch.equal(kT, hT)
    else:
        assert not kT[0].isfinite().all()
    assert not y[0, bad].isfinite().all()


def test_thousands_of_packed_sequences():
    """Nine thousand sequences of some thirty tokens, and one of many segments at the
    end: more than the sums of dB and dC had workgroups for."""
    H, P, N, G = 8, 64, 128, 8
    lens = torch.randint(0, 60, (9000,), generator=torch.Generator().manual_seed(5)).tolist() + [20000]
    n, T = len(lens), sum(lens)
    g = torch.Generator(device=DEV).manual_seed(6)
    new = lambda *s, dtype=BF: torch.randn(*s, generator=g, device=DEV, dtype=dtype)  # noqa: E731
    x, dy, B, C, dt = new(1, T, H, P), new(1, T, H, P), new(1, T, G, N), new(1, T, G, N), new(1, T, H, dtype=F32)
    A, rest = -torch.rand(H, generator=g, device=DEV) - 0.1, dict(dt_bias=torch.full((H,), -3.0, device=DEV))
    cu = offsets(lens)
    y, hT = gdn.ssm_forward(x, dt, A, B, C, **rest, cu_seqlens=cu)
    grads = gdn.ssm_backward(dy, x, dt, A, B, C, **rest, cu_seqlens=cu)
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    off = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    for k in (0, 1, 63, 64, 4999, 8998, 8999, 9000):
        s = slice(at[k], at[k + 1])
        args = [t[:, s].contiguous() for t in (x, dt)] + [A] + [t[:, s].contiguous() for t in (B, C)]
        y1, h1 = gdn.ssm_forward(*args, **rest)
        g1 = gdn.ssm_backward(dy[:, s].contiguous(), *args, **rest)
        pairs = [(y[:, s], y1), (hT[k:k + 1], h1)] + [(grads[i][:, s], g1[i]) for i in (0, 1, 3, 4)]
        assert all(torch.equal(u, v) if k < 9000 else off(u, v) < 2.0 ** -6 for u, v in pairs), k
