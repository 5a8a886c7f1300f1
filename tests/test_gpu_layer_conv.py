"""Short causal convolution on the GPU against its definition in 64 bits.

Tolerances.  v is a sum of W + 1 <= 5 terms in fp32: 6 * 2^-24 of its terms' size
S.  silu and its derivative have slopes below 1.1 and 0.6, and an exponential,
a reciprocal and two products of 2 units each: y and dv are within 2^-20 of
S (and |dy| (1.1 + S)) before they are stored (bf16 2^-8, fp32 2^-24, relative).
Sums over n tokens add at most (32 k + 80) roundings, k runs of a wave."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


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


CASES = [  # lens (None: batch of B x T), D, W, type, weights' type, bias, state, silu
    ((1, 1), 8, 4, BF, BF, True, False, True), ((2, 31), 5, 4, F32, F32, True, True, True),
    ((1, 32), 64, 3, BF, F32, False, True, False), ((3, 33), 260, 2, BF, BF, True, True, True),
    ((2, 100), 1028, 4, BF, F32, True, False, True), ((1, 257), 77, 4, BF, BF, False, False, True),
    ([5, 0, 1, 2, 3, 40, 64, 0, 33], 260, 4, BF, BF, True, True, True),
    ([0, 0, 7], 12, 4, F32, F32, True, True, True), ([200], 256, 3, F32, F32, True, False, False),
    ([1] * 70, 36, 4, BF, BF, True, True, True), ([31, 32, 33, 1, 95], 514, 2, BF, F32, True, True, True)]


@pytest.mark.parametrize("lens,D,W,dt,wt,bias,state,silu", CASES)
def test_forward_and_backward(lens, D, W, dt, wt, bias, state, silu):
    packed = isinstance(lens, list)
    B, T = (1, sum(lens)) if packed else lens
    each = lens if packed else [T] * B
    n = len(each)
    x, w = rnd(B, T, D, seed=1, dtype=dt), rnd(D, W, seed=2, dtype=wt, scale=0.5)
    b = rnd(D, seed=3, dtype=wt, scale=0.3) if bias else None
    st = rnd(n, W - 1, D, seed=4, dtype=dt) if state else None
    cu = offsets(lens) if packed else None
    act = "silu" if silu else None
    y, last = gdn.conv_forward(x, w, b, activation=act, initial_state=st, cu_seqlens=cu)
    flat = x.reshape(-1, D)
    ref, rlast = L.conv(flat, w, b, st, each, silu)
    size, _ = L.conv(flat, w, b, st, each, silu, absolute=True)
    close(y.reshape(-1, D), ref, ref.abs() * HALF[dt] + size * 2.0 ** -20, "y")
    assert torch.equal(last.cpu().double(), rlast)
    dy, df = rnd(B, T, D, seed=5, dtype=dt), rnd(n, W - 1, D, seed=6, dtype=dt)
    dx, dw, db, di = gdn.conv_backward(dy, x, w, b, activation=act, initial_state=st, cu_seqlens=cu, dfinal=df)
    assert (db is None) == (b is None) and (di is None) == (st is None)
    g = L.conv_grad(dy.reshape(-1, D), flat, w, b, st, each, silu, df)
    # dv's error is |dy| (1.1 + S) 2^-20: as sizes, dy grows by 1 + S
    a = L.conv_grad((dy.reshape(-1, D).cpu().double() * (1.1 + size)), flat, w, b, st, each, silu, df, absolute=True)
    close(dx.reshape(-1, D), g[0], g[0].abs() * HALF[dt] + a[0] * 2.0 ** -20, "dx")
    adds = (32 * 4 + 80) * 2.0 ** -24
    close(dw, g[1], a[1] * (2.0 ** -20 + adds), "dw")
    if b is not None:
        close(db, g[2], a[2] * (2.0 ** -20 + adds), "db")
    if st is not None:
        close(di, g[3], g[3].abs() * HALF[dt] + a[3] * 2.0 ** -20, "dinitial")


@pytest.mark.parametrize("D,dt", [(8, BF), (260, BF), (77, F32), (1024, BF)])
@pytest.mark.parametrize("W", [2, 4])
def test_steps_are_the_forward_pass(D, dt, W):
    """T steps give the same bits as a forward pass of T tokens, and its state."""
    B, T = 3, 6
    x, w, b = rnd(B, T, D, seed=1, dtype=dt), rnd(D, W, seed=2, dtype=dt), rnd(D, seed=3, dtype=dt)
    st = rnd(B, W - 1, D, seed=4, dtype=dt)
    y, last = gdn.conv_forward(x, w, b, initial_state=st)
    pool = torch.full((5, W - 1, D), float("nan"), device=DEV, dtype=dt)
    slots = torch.tensor([3, 0, 4], device=DEV, dtype=torch.int32)
    pool[slots.long()] = st
    for t in range(T):
        assert torch.equal(gdn.conv_step(x[:, t], pool, w, b, slots=slots), y[:, t]), t
    assert torch.equal(pool[slots.long()], last)
    assert pool[[1, 2]].isnan().all()
    direct = st.clone()
    for t in range(T):
        gdn.conv_step(x[:, t], direct, w, b)
    assert torch.equal(direct, last)


def test_step_padding_and_repeated_slots():
    B, D = 70, 36
    x, w = rnd(B, D, seed=1, dtype=BF), rnd(D, 4, seed=2, dtype=BF)
    pool = rnd(80, 3, D, seed=3, dtype=BF)
    slots = torch.randperm(80, generator=torch.Generator().manual_seed(4))[:B].to(torch.int32).to(DEV)
    slots[5], slots[6], slots[7] = -1, 80, -2 ** 31
    slots[66] = slots[2]
    slots[67] = slots[2]
    before = pool.clone()
    y = gdn.conv_step(x, pool, w, slots=slots)
    pad = [5, 6, 7, 66, 67]
    keep = [i for i in range(B) if i not in pad]
    assert y[pad].eq(0).all()
    alone = before.clone()
    ref = gdn.conv_step(x[keep], alone, w, slots=slots[keep])
    assert torch.equal(y[keep], ref) and torch.equal(pool, alone)
    assert torch.equal(gdn.conv_step(x[:0], pool, w), x[:0])


def test_rows_behind_the_sequences_and_malformed_offsets():
    D = 264
    x = rnd(1, 90, D, seed=1, dtype=BF)
    x[:, 70:] = float("nan")
    w = rnd(D, 4, seed=2, dtype=BF)
    y = torch.full_like(x, 7.0)
    cu = offsets([30, 0, 40])
    gdn.conv_forward(x, w, cu_seqlens=cu, y=y)
    ref, _ = gdn.conv_forward(x[:, :70], w, cu_seqlens=cu)
    assert torch.equal(y[:, :70], ref) and y[:, 70:].eq(7.0).all()
    dy = rnd(1, 90, D, seed=3, dtype=BF)
    dx, dw, _, _ = gdn.conv_backward(dy, x, w, cu_seqlens=cu)
    dx0, dw0, _, _ = gdn.conv_backward(dy[:, :70].contiguous(), x[:, :70].contiguous(), w, cu_seqlens=cu)
    assert torch.equal(dx[:, :70], dx0) and dx[:, 70:].eq(0).all()
    # (three runs of 32 tokens and two: the same additions, in the same places)
    assert torch.allclose(dw, dw0, rtol=0, atol=float(dw0.abs().max()) * 2.0 ** -18)
    # a first offset behind 0 leaves the rows before it alone
    y = torch.full_like(x, 7.0)
    late = torch.tensor([13, 40, 70], device=DEV, dtype=torch.int32)
    gdn.conv_forward(x, w, cu_seqlens=late, y=y)
    ref, _ = gdn.conv_forward(x[:, 13:70].contiguous(), w, cu_seqlens=late - 13)
    assert torch.equal(y[:, 13:70], ref) and y[:, :13].eq(7.0).all()
    # offsets out of range or order: wrong rows, no access outside the tensors
    for bad in ([0, 1000, 90], [-5, 40, 20, 90], [50, 10], [2 ** 31 - 1, -2 ** 31]):
        out, last = gdn.conv_forward(rnd(1, 90, D, seed=4, dtype=BF), w, cu_seqlens=torch.tensor(bad, device=DEV, dtype=torch.int32))
        gdn.conv_backward(dy, rnd(1, 90, D, seed=4, dtype=BF), w, cu_seqlens=torch.tensor(bad, device=DEV, dtype=torch.int32))
    torch.cuda.synchronize()


def test_strided_tokens():
    """x as columns of a wider buffer, aligned to four elements or not."""
    big = rnd(2, 50, 700, seed=1, dtype=BF)
    w = rnd(256, 4, seed=2, dtype=BF)
    dwide = rnd(2, 50, 600, seed=3, dtype=BF)
    for at in (64, 65):
        x, dy = big[..., at:at + 256], dwide[..., at:at + 256]
        y, last = gdn.conv_forward(x, w)
        ref, rlast = L.conv(x.reshape(-1, 256), w, None, None, [50, 50], True)
        size, _ = L.conv(x.reshape(-1, 256), w, None, None, [50, 50], True, absolute=True)
        close(y.reshape(-1, 256), ref, ref.abs() * 2.0 ** -8 + size * 2.0 ** -20, "y")
        assert torch.equal(last.cpu().double(), rlast)
        a = gdn.conv_backward(dy, x, w)
        b = gdn.conv_backward(dy.contiguous(), x.contiguous(), w)
        assert torch.equal(a[0], b[0])
    with pytest.raises(ValueError, match="contiguous behind"):
        gdn.conv_forward(big[..., ::2][..., :256], w)


def test_refused():
    x, w = rnd(2, 10, 64, seed=1), rnd(64, 4, seed=2)
    cu = offsets([20])
    for bad, err in ((lambda: gdn.conv_forward(x, rnd(64, 5, seed=1)), ValueError), (lambda: gdn.conv_forward(x, w, cu_seqlens=cu), ValueError),
                     (lambda: gdn.conv_forward(x[:1], w, cu_seqlens=cu.long()), TypeError), (lambda: gdn.conv_forward(x, w.to(BF)), TypeError),
                     (lambda: gdn.conv_forward(x, w, activation="relu"), ValueError), (lambda: gdn.conv_forward(x[0], w), ValueError),
                     (lambda: gdn.conv_forward(x, w, initial_state=x[:, :2]), ValueError), (lambda: gdn.conv_forward(x, w, y=x), ValueError),
                     (lambda: gdn.conv_step(x[0], x, w), ValueError), (lambda: gdn.conv_step(x[:, 0], rnd(1, 3, 64, seed=1), w), gdn.GdnError),
                     (lambda: gdn.conv_step(x[:, 0], rnd(2, 3, 64, seed=1), w, slots=torch.zeros(3, device=DEV, dtype=torch.int32)), ValueError),
                     (lambda: gdn.conv_forward(x[:, :1].expand(2, 5, 64).transpose(0, 1)[:, :1], w[:32]), ValueError)):
        with pytest.raises(err):
            bad()
    y, last = gdn.conv_forward(x[:, :0], w)
    assert y.shape == (2, 0, 64) and last.eq(0).all()
    dx, dw, _, _ = gdn.conv_backward(x[:, :0], x[:, :0], w)
    assert dw.eq(0).all()


def test_gradient_against_differences():
    """fp32: as for the norm, a difference over 2 h, h = 2^-8, of a loss known to
    2^-20 of its terms, and a third derivative below 1 in the same sizes."""
    lens, D, W, h = [40, 3, 60], 64, 4, 2.0 ** -8
    x, w, b, st = rnd(1, 103, D, seed=1), rnd(D, W, seed=2, scale=0.5), rnd(D, seed=3), rnd(3, W - 1, D, seed=4)
    dy, df, cu = rnd(1, 103, D, seed=5), rnd(3, W - 1, D, seed=6), offsets(lens)

    def loss(x, w, b, st):
        y, last = gdn.conv_forward(x, w, b, initial_state=st, cu_seqlens=cu)
        return (y.double() * dy.double()).sum() + (last.double() * df.double()).sum()

    g = gdn.conv_backward(dy, x, w, b, initial_state=st, cu_seqlens=cu, dfinal=df)
    size, _ = L.conv(x[0], w, b, st, lens, True, absolute=True)
    terms = float(((1 + size) * dy[0].cpu().double().abs()).sum() + df.abs().double().sum())
    leaves = [x, w, b, st]
    for i in range(4):
        d = rnd(*leaves[i].shape, seed=20 + i)
        plus, minus = list(leaves), list(leaves)
        plus[i], minus[i] = leaves[i] + h * d, leaves[i] - h * d
        num = float((loss(*plus) - loss(*minus)) / (2 * h))
        assert abs(num - float((g[i].double() * d.double()).sum())) <= terms * 2.0 ** -10, i


def test_long_rows_pass_32_bit_offsets():
    """Two batches of 2.1 * 2^30 bytes each: a row's place needs 33 bits."""
    T, D = 140000, 8192
    x = torch.empty(2, T, D, device=DEV, dtype=BF).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    w = rnd(D, 4, seed=2, dtype=BF)
    y, last = gdn.conv_forward(x, w)
    for b in (0, 1):
        part, _ = gdn.conv_forward(x[b:b + 1, T - 64:], w)
        assert torch.equal(y[b, T - 61:], part[0, 3:]), b
        assert torch.equal(last[b], x[b, T - 3:])
    del y
    dx, _, _, _ = gdn.conv_backward(x, x, w)
    part = gdn.conv_backward(x[1:, T - 64:], x[1:, T - 64:], w)[0]
    assert torch.equal(dx[1, T - 61:], part[0, 3:])


def test_streams_graphs_and_repeats():
    x, w, b, dy = rnd(2, 300, 512, seed=1, dtype=BF), rnd(512, 4, seed=2, dtype=BF), rnd(512, seed=3, dtype=BF), rnd(2, 300, 512, seed=4, dtype=BF)
    pool0 = rnd(4, 3, 512, seed=5, dtype=BF)
    slots = torch.tensor([2, 0], device=DEV, dtype=torch.int32)
    pool = pool0.clone()

    def work():
        pool.copy_(pool0)
        y, last = gdn.conv_forward(x, w, b, initial_state=pool[:2])
        return [y, last, gdn.conv_step(x[:, 7], pool, w, b, slots=slots), *gdn.conv_backward(dy, x, w, b)[:3]]

    ref = [t.clone() for t in work()]
    assert all(torch.equal(a, c) for a, c in zip(ref, work()))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, _ = gdn.conv_forward(x, w, b, initial_state=pool0[:2], stream=st)
    st.synchronize()
    assert torch.equal(y, ref[0])
    with torch.cuda.stream(st):
        work()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = work()
    for k in range(3):
        x.copy_(rnd(2, 300, 512, seed=10 + k, dtype=BF))
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, c) for a, c in zip(kept, work())), k


def test_slots_behind_32_bit_offsets():
    S, D, W = 90000, 8192, 4
    pool = torch.zeros(S, W - 1, D, device=DEV, dtype=BF)
    assert pool.numel() * 2 > 1 << 32
    x, w, st = rnd(3, D, seed=1, dtype=BF), rnd(D, W, seed=2, dtype=BF), rnd(3, W - 1, D, seed=3, dtype=BF)
    slots = torch.tensor([S - 1, 7, 88000], device=DEV, dtype=torch.int32)
    pool[slots.long()] = st
    y = gdn.conv_step(x, pool, w, slots=slots)
    ref = gdn.conv_step(x, st, w)
    assert torch.equal(y, ref) and torch.equal(pool[slots.long()], st)
