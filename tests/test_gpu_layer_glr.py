"""The gated linear recurrence on the GPU against the recurrence in 64 bits.

Tolerances are the oracle's (oracle/layer.py, glr): the errors that fp32 states,
gates and sums may have, token by token, plus half a step of the type that a
result is stored in (bf16 2^-8, fp32 2^-24)."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = 2.0 ** -120         # the smallest exponentials are zeros


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def close(got, ref, err, what):
    d = (got.detach().cpu().double() - ref).abs()
    tol = err + ref.abs() * HALF[got.dtype] + TINY
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e over its tolerance" % (what, int(bad.sum()), bad.numel(),
                                                                               float((d - tol).max()))


def gates(*shape, form, seed, dtype, memory=20.0):
    """Raw gates, bias and rate of decays whose memories are around ``memory`` tokens."""
    D = shape[-1]
    raw = rnd(*shape, seed=seed)
    if form == "log":
        return (torch.nn.functional.logsigmoid(raw) / memory).to(dtype), None, None
    u = torch.rand(D, generator=torch.Generator().manual_seed(seed + 1)).to(DEV)
    if form == "sigmoid":
        return raw.to(dtype), torch.log(torch.tensor(memory, device=DEV)) * (0.5 + u), None
    return raw.to(dtype), 0.3 * rnd(D, seed=seed + 2), (0.5 + u) * 2 / memory


def inputs(B, T, D, dt, gt, form, seed=1, memory=20.0, n=None, h0=True):
    gate, bias, rate = gates(B, T, D, form=form, seed=seed, dtype=gt, memory=memory)
    d = dict(x=rnd(B, T, D, seed=seed + 10, dtype=dt), gate=gate, gate_bias=bias, rate=rate,
             h0=rnd(n or B, D, seed=seed + 11) if h0 else None)
    d["dy"], d["dhT"] = rnd(B, T, D, seed=seed + 12, dtype=dt), rnd(n or B, D, seed=seed + 13) if h0 else None
    return d


def reference(d, lens, form, scale, grads=True):
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    return L.glr(flat(d["x"]), flat(d["gate"]), d["gate_bias"], d["rate"], d["h0"], lens, form, scale,
                 flat(d["dy"]) if grads else None, d["dhT"] if grads else None)


def check(d, lens, form, scale, cu=None, grads=True, **out):
    """Forward and backward of inputs d against the oracle; returns the results."""
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form=form, scale=scale, cu_seqlens=cu)
    ref = reference(d, lens, form, scale, grads)
    rows = slice(0, sum(lens))
    y, hT = gdn.glr_forward(d["x"], d["gate"], d["h0"], **kw)
    close(y.flatten(0, 1)[rows], ref["y"][rows], ref["y_err"][rows], "y")
    close(hT, ref["hT"], ref["hT_err"], "hT")
    if not grads:
        return [y, hT]
    dx, dg, db, dr, dh0 = gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], **kw, **out)
    close(dx.flatten(0, 1)[rows], ref["dx"][rows], ref["dx_err"][rows], "dx")
    close(dg.flatten(0, 1)[rows], ref["dgate"][rows], ref["dgate_err"][rows], "dgate")
    for name, v, of in (("dbias", db, d["gate_bias"]), ("drate", dr, d["rate"]), ("dh0", dh0, d["h0"])):
        assert (v is None) == (of is None), name
        if v is not None:
            close(v, ref[name], ref[name + "_err"], name)
    return [y, hT, dx, dg, db, dr, dh0]


FORMS = list(itertools.product(("log", "sigmoid", "rate"), (None, "complement", "norm")))
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("form,scale", FORMS)
@pytest.mark.parametrize("dt,gt", TYPES)
def test_forms_and_types(form, scale, dt, gt):
    check(inputs(2, 150, 66, dt, gt, form), [150, 150], form, scale)


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("D,dt", [(64, BF), (63, BF), (130, F32)])
def test_lengths(T, D, dt):
    for form, scale, h0 in (("rate", "norm", True), ("sigmoid", "complement", False)):
        check(inputs(1, T, D, dt, dt, form, h0=h0), [T], form, scale)


@pytest.mark.parametrize("T", [1, 5, 16, 33, 64])
@pytest.mark.parametrize("D,dt", [(66, BF), (65, BF), (64, F32)])
def test_many_short_sequences(T, D, dt):
    """A wave each: over a thousand of them."""
    B = 700
    check(inputs(B, T, D, dt, dt, "rate"), [T] * B, "rate", "norm")


@pytest.mark.parametrize("T,D,dt", [(70, 66, BF), (130, 65, BF), (65, 130, F32)])
def test_many_sequences_of_some_tiles(T, D, dt):
    """Four waves each."""
    B = 520
    check(inputs(B, T, D, dt, dt, "sigmoid"), [T] * B, "sigmoid", "complement", grads=False)


def test_growing_states():
    """Gates above zero: the state grows, by a tenth a token at most here."""
    d = inputs(1, 200, 64, F32, F32, "log")
    d["gate"] = d["gate"].abs().clamp(max=0.1) * torch.where(rnd(1, 200, 64, seed=3) > 0, 1.0, -1.0)
    for scale in (None, "complement"):
        check(d, [200], "log", scale)


@pytest.mark.parametrize("D", [1, 2, 3, 62, 64, 65, 128, 200])
@pytest.mark.parametrize("dt", [BF, F32])
def test_widths(D, dt):
    check(inputs(3, 40, D, dt, dt, "rate"), [40] * 3, "rate", "norm")


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("form,scale,memory", [("rate", "norm", 1000.0), ("sigmoid", "complement", 3000.0), ("log", None, 300.0),
                                               ("log", "norm", 2.0)])
def test_segments_and_long_memories(dt, gt, form, scale, memory):
    """Several segments, and memories as long as all of them: the last state still holds the first."""
    d = inputs(1, 4500, 6, dt, gt, form, memory=memory)
    _, hT, *_ = check(d, [4500], form, scale)
    if memory >= 1000:
        ref = L.glr(d["x"][0], d["gate"][0], d["gate_bias"], d["rate"], d["h0"], [4500], form, scale)["hT"]
        assert (hT.cpu().double() - ref).norm() <= 1e-6 * ref.norm()


@pytest.mark.parametrize("lens,packed", [([9100], False), ([9100, 9100], False), ([3000, 0, 4100, 1, 1999], True)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_segments_in_uneven_pieces(lens, packed, dt):
    """Wide enough that a segment's move is put together from a few pieces of some tiles; the
    recurrence of single channels is compared in some of them, the first and the last among them."""
    B = 1 if packed else len(lens)
    D = 4100 // B
    d = inputs(B, sum(lens) if packed else lens[0], D, dt, dt, "sigmoid", n=len(lens), memory=500.0)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV) if packed else None
    y, hT = gdn.glr_forward(d["x"], d["gate"], d["h0"], gate_bias=d["gate_bias"], form="sigmoid", scale="complement", cu_seqlens=cu)
    cols = [0, 1, 63, 64, 1027, D - 1]
    ref = reference({k: v if v is None else v[..., cols] for k, v in d.items()}, lens, "sigmoid", "complement", grads=False)
    close(y.flatten(0, 1)[:, cols], ref["y"], ref["y_err"], "y")
    close(hT[:, cols], ref["hT"], ref["hT_err"], "hT")


@pytest.mark.parametrize("lens", [[1], [0, 5], [5, 0, 0, 70, 1, 0, 300, 16, 2], [3] * 70, [0, 0, 0], [600, 1, 1, 1, 700, 0], [256, 256, 256, 128],
                                  [1300, 0, 2200]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_packed_sequences(lens, dt):
    """Every sequence is what it is alone; rows behind the last and before the first stay as they were."""
    front, behind = 7, 9
    n, T = len(lens), sum(lens)
    form, scale = "rate", "norm"
    d = inputs(1, T, 34, dt, dt, form, n=n)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    whole = check(d, lens, form, scale, cu=cu)
    pad = lambda t, v: torch.cat([torch.full((1, front, 34), v, device=DEV, dtype=dt), t,  # noqa: E731
                                  torch.full((1, behind, 34), v, device=DEV, dtype=dt)], 1)
    nan = float("nan")
    y, hT = pad(torch.zeros_like(whole[0]), 5.0), torch.empty_like(whole[1])
    x, gate, dy = pad(d["x"], nan), pad(d["gate"], nan), pad(d["dy"], nan)
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form=form, scale=scale, cu_seqlens=cu + front)
    gdn.glr_forward(x, gate, d["h0"], y=y, hT=hT, **kw)
    dx, dg = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    more = gdn.glr_backward(dy, x, gate, d["h0"], d["dhT"], dx=dx, dgate=dg, **kw)
    at = slice(front, front + T)
    for got, want in ((y, whole[0]), (dx, whole[2]), (dg, whole[3])):
        assert got[:, :front].eq(5.0).all() and got[:, front + T:].eq(5.0).all()
        assert (got[:, at].float() - want.float()).abs().max() <= (want.float().abs().max() * 2.0 ** -7 if T else 0) if T else True
    # (in other places of the tiles: other orders of the same sums)
    ref = reference(d, lens, form, scale)
    close(y[0, at], ref["y"], ref["y_err"], "y, shifted")
    close(hT, ref["hT"], ref["hT_err"], "hT, shifted")
    close(dx[0, at], ref["dx"], ref["dx_err"], "dx, shifted")
    close(dg[0, at], ref["dgate"], ref["dgate_err"], "dgate, shifted")
    for name, v in (("dbias", more[2]), ("drate", more[3]), ("dh0", more[4])):
        close(v, ref[name], ref[name + "_err"], name + ", shifted")


def test_what_a_nan_reaches():
    """Its own sequence and channel from its token on (y), up to it (dx); nothing of another's."""
    lens = [200, 300, 40]
    d = inputs(1, 540, 64, F32, F32, "sigmoid", n=3)
    cu = torch.tensor([0, 200, 500, 540], dtype=torch.int32, device=DEV)
    kw = dict(gate_bias=d["gate_bias"], form="sigmoid", scale="complement", cu_seqlens=cu)
    y0, h0 = gdn.glr_forward(d["x"], d["gate"], d["h0"], **kw)
    g0 = gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], **kw)
    for bad in (float("nan"), float("inf")):
        x, dy = d["x"].clone(), d["dy"].clone()
        x[0, 320, 5] = bad
        y, hT = gdn.glr_forward(x, d["gate"], d["h0"], **kw)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, 320:500, 5] = True
        assert not y[hit].isfinite().any() and torch.equal(y[~hit], y0[~hit])
        assert not hT[1, 5].isfinite() and hT.isfinite().sum() == hT.numel() - 1 and torch.equal(hT[::2], h0[::2])
        dx, dg, _, _, dh0 = gdn.glr_backward(d["dy"], x, d["gate"], d["h0"], d["dhT"], **kw)
        assert torch.equal(dx, g0[0])                        # dx does not read x
        hit[0, 320, 5] = True
        assert torch.equal(dg[~hit], g0[1][~hit]) and torch.equal(dh0, g0[4])
        dy[0, 320, 5] = bad
        dx, dg, _, _, dh0 = gdn.glr_backward(dy, d["x"], d["gate"], d["h0"], d["dhT"], **kw)
        hit = torch.zeros_like(hit)
        hit[0, 200:321, 5] = True
        assert not dx[hit].isfinite().any() and torch.equal(dx[~hit], g0[0][~hit]) and torch.equal(dg[~hit], g0[1][~hit])
        assert dh0.isfinite().sum() == dh0.numel() - 1


def test_extreme_gates():
    """Decays of exactly 1 and 0: the state stays or goes."""
    T, D = 300, 64
    d = inputs(1, T, D, F32, F32, "log")
    inf = float("inf")
    for form, keep, drop, scale in (("log", 0.0, -inf, None), ("log", 0.0, -inf, "norm"), ("log", 0.0, -200.0, "complement"),
                                    ("sigmoid", inf, -inf, "complement"), ("sigmoid", 300.0, -300.0, "norm"), ("rate", -inf, inf, "norm"),
                                    ("rate", -300.0, 300.0, "complement")):
        gate = torch.full((1, T, D), keep, device=DEV)
        gate[0, 100::50] = drop
        rate = torch.full((D,), 300.0, device=DEV) if form == "rate" else None
        kw = dict(rate=rate, form=form, scale=scale)
        y, hT = gdn.glr_forward(d["x"], gate, d["h0"], **kw)
        a, _, k, _, _, _ = L.glr_gates(gate[0], None, rate, form, scale)
        assert ((a == 1) | (a < 1e-80)).all()
        h, want = L.f64(d["h0"][0]), torch.zeros(T, D, dtype=torch.float64)
        for t in range(T):
            h = a[t] * h + k[t] * L.f64(d["x"][0, t])
            want[t] = h
        close(y[0], want, (want.abs() + 64) * 2.0 ** -18, (form, scale))
        got = gdn.glr_backward(d["dy"], d["x"], gate, d["h0"], d["dhT"], **kw)
        assert all(t is None or t.isfinite().all() for t in got), (form, scale)
        dh, dx = L.f64(d["dhT"][0]), torch.zeros(T, D, dtype=torch.float64)
        for t in reversed(range(T)):
            dh = dh + L.f64(d["dy"][0, t])
            dx[t], dh = k[t] * dh, a[t] * dh
        close(got[0][0], dx, (dx.abs() + 64) * 2.0 ** -18, (form, scale, "dx"))


def test_strided_tensors_and_parts_of_one_buffer():
    B, T, D = 2, 300, 64
    d = inputs(B, T, D, BF, BF, "rate")
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form="rate", scale="norm")
    want = gdn.glr_forward(d["x"], d["gate"], d["h0"], **kw)
    grads = gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], **kw)
    for first, width in ((0, 2 * D), (2, 2 * D + 10), (1, 2 * D + 3)):          # aligned, and not to two elements
        both = torch.full((B, T, width), 3.0, device=DEV, dtype=BF)
        x, gate = both[..., first:first + D], both[..., first + D:first + 2 * D]
        x.copy_(d["x"])
        gate.copy_(d["gate"])
        y, hT = gdn.glr_forward(x, gate, d["h0"], **kw)
        out = torch.full_like(both, 3.0)
        wide = torch.zeros(T, B, 2 * D, device=DEV, dtype=BF).transpose(0, 1)[..., D:]
        wide.copy_(d["dy"])
        dx, dg = out[..., first:first + D], out[..., first + D:first + 2 * D]
        got = gdn.glr_backward(wide, x, gate, d["h0"], d["dhT"], dx=dx, dgate=dg, **kw)
        assert out[..., :first].eq(3.0).all() and out[..., first + 2 * D:].eq(3.0).all()
        if first % 2 == 0:
            assert torch.equal(y, want[0]) and torch.equal(hT, want[1])
            assert all(torch.equal(a, b) for a, b in zip(got, grads))
        else:                                   # other runs and tiles: other orders of the same sums
            ref = reference(d, [T] * B, "rate", "norm")
            for v, name in ((y.flatten(0, 1), "y"), (hT, "hT"), (dx.flatten(0, 1), "dx"), (dg.flatten(0, 1), "dgate"), (got[2], "dbias"),
                            (got[3], "drate"), (got[4], "dh0")):
                close(v, ref[name], ref[name + "_err"], name)
    # one gate for all tokens, as constant decays have it
    flat = d["gate"][:, :1].expand(B, T, D)
    a, b = gdn.glr_forward(d["x"], flat, **kw), gdn.glr_forward(d["x"], flat.contiguous(), **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("form,scale", FORMS)
def test_steps(dt, gt, form, scale):
    """A prompt, then token by token in a pool of slots: the recurrence of all of it; padding
    and rows that repeat a slot move nothing."""
    B, T, D, S = 5, 6, 300, 9
    d = inputs(B, T, D, dt, gt, form)
    pool = rnd(S, D, seed=50)
    slots = torch.tensor([4, 0, 7, 4, -1], dtype=torch.int32, device=DEV)          # row 3 repeats row 0's
    live = [0, 1, 2]
    at = slots[live].long()
    pool[at] = d["h0"][live]
    keep = pool.clone()
    ref = reference({k: None if v is None else v[live] if k in ("x", "gate", "h0", "dy", "dhT") else v for k, v in d.items()}, [T] * 3,
                    form, scale, False)
    for t in range(T):
        y = gdn.glr_step(d["x"][:, t], d["gate"][:, t], pool, gate_bias=d["gate_bias"], rate=d["rate"], form=form, scale=scale, slots=slots)
        close(y[live], ref["y"].view(3, T, D)[:, t], ref["y_err"].view(3, T, D)[:, t], t)
        assert not y[3:].float().any()
    close(pool[at], ref["hT"], ref["hT_err"], "pool")
    rest = [i for i in range(S) if i not in at.tolist()]
    assert torch.equal(pool[rest], keep[rest])
    own = d["h0"].clone()                        # without slots: row b has state b
    y = gdn.glr_step(d["x"][:, 0], d["gate"][:, 0], own, gate_bias=d["gate_bias"], rate=d["rate"], form=form, scale=scale)
    one = {k: v[:, :1] if k in ("x", "gate", "dy") else v for k, v in d.items()}
    ref = reference(one, [1] * B, form, scale, False)
    close(y, ref["y"], ref["y_err"], "y of the first token")
    close(own, ref["hT"], ref["hT_err"], "states behind it")


def test_steps_behind_32_bit_offsets():
    D, S = 1 << 15, (1 << 15) + 40               # a pool of 2^30 values and more
    pool = torch.zeros(S, D, device=DEV)
    slots = torch.tensor([S - 1, 3, S - 20], dtype=torch.int32, device=DEV)
    x, gate = rnd(3, D, seed=1), -rnd(3, D, seed=2).abs()
    pool[slots.long()] = rnd(3, D, seed=3)
    want = torch.exp(gate.double()) * pool[slots.long()].double() + x.double()
    y = gdn.glr_step(x, gate, pool, slots=slots)
    assert (y.double() - want).abs().max() <= 2.0 ** -20 * float(want.abs().max())
    assert torch.equal(pool[slots.long()], y) and int(pool.count_nonzero(1).ne(0).sum()) == 3


def test_rows_behind_32_bit_offsets():
    """Batches and tokens past 2^32 bytes are what they are alone."""
    B, T, D = 3, 5000, 1 << 17                   # 2.6 GB of x a batch in fp32, 3.9 GB in all of bf16
    x = torch.empty(B, T, D, device=DEV, dtype=BF).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    gate = torch.empty(T, D, device=DEV, dtype=BF).normal_(generator=torch.Generator(device=DEV).manual_seed(2)).neg_().abs_().neg_()
    gate = gate.expand(B, T, D)
    y, hT = gdn.glr_forward(x, gate, scale="complement")
    dx, dg, _, _, _ = gdn.glr_backward(y, x, gate, scale="complement")
    last = slice(D - 64, D)
    one = [t[2:, :, last].contiguous() for t in (x, gate, y)]
    y1, h1 = gdn.glr_forward(one[0], one[1], scale="complement")
    dx1, dg1, _, _, _ = gdn.glr_backward(one[2], one[0], one[1], scale="complement")
    # (alone its tokens are in other segments: other orders of the same sums, then rounded to bf16)
    for a, b in ((y[2:, :, last], y1), (dx[2:, :, last], dx1), (dg[2:, :, last], dg1)):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * float(b.float().abs().max())
    assert (hT[2:, last] - h1).abs().max() <= 2.0 ** -18 * float(h1.abs().max())


def test_many_states_and_sequences():
    n = 3000
    lens = [(7 * i) % 5 for i in range(n)]
    T = sum(lens)
    d = inputs(1, T, 64, BF, BF, "sigmoid", n=n)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    check(d, lens, "sigmoid", "complement", cu=cu)


def test_offsets_that_make_no_sense_stay_inside():
    """cu_seqlens is device memory: any offsets are clamped, nothing outside is touched."""
    d = inputs(1, 500, 64, BF, BF, "rate", n=4)
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form="rate", scale="norm")
    for cu in ([-5, 100, 50, 10000, 3], [500, 400, 300, 200, 100], [2 ** 31 - 1, -2 ** 31, 7, 7, 7], [0, 0, 0, 0, 0]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        guard = torch.full((3, 500, 64), 9.0, device=DEV, dtype=BF)
        gdn.glr_forward(d["x"], d["gate"], d["h0"], cu_seqlens=c, y=guard[1:2], **kw)
        assert guard[0].eq(9.0).all() and guard[2].eq(9.0).all()
        gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], cu_seqlens=c, dx=guard[1:2], **kw)
        assert guard[0].eq(9.0).all() and guard[2].eq(9.0).all()


def test_gradients_against_differences():
    """fp32, along a direction of each input: the loss's terms are known to the oracle's
    errors, here below 2^-16 of them, a difference over 2 * 2^-7 so to 2^-9; the cube's
    term is below (2^-7)^2 of the terms' sizes times a few tens."""
    d = inputs(2, 80, 64, F32, F32, "rate", memory=8.0)
    h = 2.0 ** -7
    for scale in (None, "complement", "norm"):
        grads = gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], gate_bias=d["gate_bias"], rate=d["rate"], form="rate",
                                 scale=scale)

        def loss(**new):
            v = {**d, **new}
            y, hT = gdn.glr_forward(v["x"], v["gate"], v["h0"], gate_bias=v["gate_bias"], rate=v["rate"], form="rate", scale=scale)
            return (y.double() * d["dy"].double()).sum() + (hT.double() * d["dhT"].double()).sum()

        y, hT = gdn.glr_forward(d["x"].abs(), d["gate"], d["h0"].abs(), gate_bias=d["gate_bias"], rate=d["rate"], form="rate", scale=scale)
        terms = float((y * d["dy"].abs()).double().sum() + (hT * d["dhT"].abs()).double().sum())
        for name, g in zip(("x", "gate", "gate_bias", "rate", "h0"), grads):
            way = rnd(*d[name].shape, seed=77) * (d[name] if name == "rate" else 1.0)
            num = (loss(**{name: d[name] + h * way}) - loss(**{name: d[name] - h * way})) / (2 * h)
            assert abs(float(num - (g.double() * way.double()).sum())) <= terms * 2.0 ** -8, (scale, name)


def test_streams_graphs_and_repeats():
    d = inputs(1, 3000, 192, BF, BF, "rate", n=3)
    cu = torch.tensor([0, 1500, 1501, 3000], dtype=torch.int32, device=DEV)
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form="rate", scale="norm")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    pool0 = rnd(4, 192, seed=9)

    def work():
        pool = pool0.clone()
        y = gdn.glr_step(d["x"][0, :3], d["gate"][0, :3], pool, slots=slots, **kw)
        return [y, pool, *gdn.glr_forward(d["x"], d["gate"], d["h0"], cu_seqlens=cu, **kw), *gdn.glr_forward(d["x"], d["gate"], **kw),
                *gdn.glr_backward(d["dy"], d["x"], d["gate"], d["h0"], d["dhT"], cu_seqlens=cu, **kw)]

    ref = [t.clone() for t in work()]
    assert all(torch.equal(a, b) for a, b in zip(ref, work()))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, hT = gdn.glr_forward(d["x"], d["gate"], d["h0"], cu_seqlens=cu, stream=st, **kw)
    st.synchronize()
    assert torch.equal(y, ref[2]) and torch.equal(hT, ref[3])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        d["x"].copy_(rnd(1, 3000, 192, seed=30 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, work())), k


def test_final_state_does_not_change_y():
    d = inputs(1, 3000, 64, BF, BF, "rate")
    kw = dict(gate_bias=d["gate_bias"], rate=d["rate"], form="rate", scale="norm")
    a, h = gdn.glr_forward(d["x"], d["gate"], d["h0"], **kw)
    b, none = gdn.glr_forward(d["x"], d["gate"], d["h0"], output_final_state=False, **kw)
    assert none is None and torch.equal(a, b)
    # and two halves are the whole, up to the order of sums
    y1, h1 = gdn.glr_forward(d["x"][:, :1234], d["gate"][:, :1234], d["h0"], **kw)
    y2, h2 = gdn.glr_forward(d["x"][:, 1234:], d["gate"][:, 1234:], h1, **kw)
    assert (h2 - h).abs().max() <= 2.0 ** -18 * float(h.abs().max())
    assert (torch.cat([y1, y2], 1).float() - a.float()).abs().max() <= 2.0 ** -7 * float(a.float().abs().max())


def test_refusals():
    d = inputs(2, 5, 64, F32, F32, "log")
    x, g, h0, rate = d["x"], d["gate"], d["h0"], torch.ones(64, device=DEV)
    buf = torch.empty(2, 5, 100, device=DEV)
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    pool = torch.zeros(4, 64, device=DEV)
    for bad, err in ((lambda: gdn.glr_forward(x, g[:1]), ValueError), (lambda: gdn.glr_forward(x, g.to(BF)), TypeError),
                     (lambda: gdn.glr_forward(x[0], g[0]), ValueError), (lambda: gdn.glr_forward(x, g, h0[:1]), ValueError),
                     (lambda: gdn.glr_forward(x, g, form="exp"), ValueError), (lambda: gdn.glr_forward(x, g, scale="none"), ValueError),
                     (lambda: gdn.glr_forward(x, g, form="rate"), ValueError), (lambda: gdn.glr_forward(x, g, rate=rate), ValueError),
                     (lambda: gdn.glr_forward(x, g, gate_bias=rate.to(BF)), TypeError), (lambda: gdn.glr_forward(x, g, y=x), ValueError),
                     (lambda: gdn.glr_forward(x, g, cu_seqlens=cu), ValueError), (lambda: gdn.glr_forward(x.half(), g.half()), TypeError),
                     (lambda: gdn.glr_forward(x[..., ::2], g[..., ::2]), ValueError),
                     (lambda: gdn.glr_forward(x, g, workspace=torch.empty(0, device="cpu")), ValueError),
                     (lambda: gdn.glr_backward(x, x, g, dbias=rate), ValueError), (lambda: gdn.glr_backward(x, x, g, drate=rate), ValueError),
                     (lambda: gdn.glr_backward(x, x, g, dh0=h0), ValueError), (lambda: gdn.glr_backward(x[:1], x, g), ValueError),
                     (lambda: gdn.glr_backward(x, x, g, dx=buf[..., :64], dgate=buf[..., 36:]), ValueError),
                     (lambda: gdn.glr_backward(x, x, g, dx=buf[:, :1, :64].expand(2, 5, 64)), ValueError),
                     (lambda: gdn.glr_step(x[:, 0], g[:, 0], pool[:1]), gdn.GdnError), (lambda: gdn.glr_step(x[:, 0], g[:, 0], pool[0]), ValueError),
                     (lambda: gdn.glr_step(x[:, 0], g[:, 0], pool.to(BF)), TypeError), (lambda: gdn.glr_step(pool[:2], g[:, 0], pool), ValueError),
                     (lambda: gdn.glr_step(x[:, 0], g[:, 0], pool, slots=cu.long()), TypeError)):
        with pytest.raises(err):
            bad()
