"""A block of the gated linear recurrence, its operators run together as a layer uses
them: layer norm with the residual's addition, projection, recurrence, gated norm,
projection; prompts in one call, in two, and token by token from the pool; and a
training step through all of them against 64-bit autograd of the same formulas."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DM, H, P = 96, 3, 64
D = H * P
FORM = dict(form="rate", scale="norm")


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def weights(dtype):
    return dict(norm=(1 + rnd(DM, seed=1, scale=0.1)).to(dtype), nbias=rnd(DM, seed=2, dtype=dtype, scale=0.1),
                w_in=rnd(DM, 3 * D, seed=3, dtype=dtype, scale=DM ** -0.5), bias=rnd(D, seed=4), rate=rnd(D, seed=5).abs() * 0.1 + 0.01,
                gnorm=(1 + rnd(H, P, seed=6, scale=0.1)).to(dtype), w_out=rnd(D, DM, seed=7, dtype=dtype, scale=D ** -0.5))


def gates(w):
    return dict(gate_bias=w["bias"], rate=w["rate"], **FORM)


def heads(t):
    return t.unflatten(-1, (H, P))


def prompt(w, x, res, state=None, cu=None):
    y, s, _ = gdn.layer_norm_forward(x, w["norm"], w["nbias"], res)
    z = y @ w["w_in"]                            # x, the recurrence's gate and the norm's, side by side
    h, state = gdn.glr_forward(z[..., :D], z[..., D:2 * D], state, cu_seqlens=cu, **gates(w))
    o = gdn.gate_norm_forward(heads(h), heads(z[..., 2 * D:]), w["gnorm"])
    return o.flatten(-2) @ w["w_out"], s, state


def token(w, x, res, pool, slots):
    y, s, _ = gdn.layer_norm_forward(x, w["norm"], w["nbias"], res)
    z = y @ w["w_in"]
    h = gdn.glr_step(z[..., :D], z[..., D:2 * D], pool, slots=slots, **gates(w))
    o = gdn.gate_norm_forward(heads(h), heads(z[..., 2 * D:]), w["gnorm"])
    return o.flatten(-2) @ w["w_out"], s


def test_prompt_then_tokens_is_one_prompt():
    """fp32: the same numbers by three ways.  Each value is a sum of at most a few
    hundred products in fp32, in another order each way: 2^-13 of the largest."""
    w, lens, k = weights(F32), [40, 330, 7], 5
    x, res = rnd(1, sum(lens), DM, seed=10), rnd(1, sum(lens), DM, seed=11)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    o, s, hT = prompt(w, x, res, cu=cu)
    tol = float(o.abs().max()) * 2.0 ** -13
    # the first tokens of each as one packed prompt, the last five one by one
    rows = torch.cat([torch.arange(n - k) + int(b) for n, b in zip(lens, cu[:-1])]).to(DEV)
    cu2 = torch.tensor([0] + [n - k for n in lens]).cumsum(0).to(torch.int32).to(DEV)
    o2, _, h2 = prompt(w, x[:, rows].contiguous(), res[:, rows].contiguous(), cu=cu2)
    assert (o[:, rows] - o2).abs().max() <= tol
    pool = rnd(6, D, seed=13)
    slots = torch.tensor([4, 1, 5, -1], device=DEV, dtype=torch.int32)       # the last row is padding
    pool[slots[:3].long()] = h2
    for t in range(k):
        at = torch.tensor([int(b) + n - k + t for n, b in zip(lens, cu[:-1])], device=DEV)
        ot, st = token(w, torch.cat([x[0, at], x[0, :1]]), torch.cat([res[0, at], res[0, :1]]), pool, slots)
        assert (ot[:3] - o[0, at]).abs().max() <= tol, t
        assert torch.equal(st[:3], s[0, at])
    assert (pool[slots[:3].long()] - hT).abs().max() <= float(hT.abs().max()) * 2.0 ** -13


def plain(w, x, res):
    """The block's formulas in 64 bits, token by token."""
    s = x + res
    y = torch.nn.functional.layer_norm(s, (DM,), w["norm"], w["nbias"], 1e-5)
    z = y @ w["w_in"]
    a = torch.exp(-w["rate"] * torch.sigmoid(z[..., D:2 * D] + w["bias"]))
    u = torch.sqrt(1 - a * a) * z[..., :D]
    h, out = torch.zeros(x.shape[0], D, dtype=x.dtype), []
    for t in range(x.shape[1]):
        h = a[:, t] * h + u[:, t]
        out.append(h)
    n = heads(torch.stack(out, 1))
    n = n * (n.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w["gnorm"] * torch.nn.functional.silu(heads(z[..., 2 * D:]))
    return n.flatten(-2) @ w["w_out"], s


def test_training_step_through_the_block():
    """fp32: gradients of all weights and inputs against 64-bit autograd.  Each way
    through the block is a few hundred fp32 roundings of sums of both signs: each
    gradient within 2^-11 of its own norm."""
    w, B, T = weights(F32), 2, 90
    x, res, do, ds = (rnd(B, T, DM, seed=20 + i) for i in range(4))
    y, s, _ = gdn.layer_norm_forward(x, w["norm"], w["nbias"], res)
    z = y @ w["w_in"]
    h, _ = gdn.glr_forward(z[..., :D], z[..., D:2 * D], **gates(w))
    o = gdn.gate_norm_forward(heads(h), heads(z[..., 2 * D:]), w["gnorm"])
    got = {"w_out": o.flatten(0, 1).flatten(1).T @ do.flatten(0, 1)}
    # every gradient goes straight to its place in the projection's
    dz = torch.empty(B, T, 3 * D, device=DEV)
    dh, _, got["gnorm"], _ = gdn.gate_norm_backward(heads(do @ w["w_out"].T), heads(h), heads(z[..., 2 * D:]), w["gnorm"], dz=heads(dz[..., 2 * D:]))
    _, _, got["bias"], got["rate"], _ = gdn.glr_backward(dh.flatten(-2), z[..., :D], z[..., D:2 * D], dx=dz[..., :D], dgate=dz[..., D:2 * D],
                                                         **gates(w))
    got["w_in"] = y.flatten(0, 1).T @ dz.flatten(0, 1)
    got["x"], _, got["norm"], got["nbias"] = gdn.layer_norm_backward(dz @ w["w_in"].T, s, w["norm"], w["nbias"], ds)
    leaves = {k: v.detach().cpu().double().requires_grad_() for k, v in {**w, "x": x}.items()}
    out, kept = plain(leaves, leaves["x"], res.cpu().double())
    ((out * do.cpu().double()).sum() + (kept * ds.cpu().double()).sum()).backward()
    for k, v in got.items():
        ref = leaves[k].grad
        assert (v.cpu().double() - ref).norm() <= ref.norm() * 2.0 ** -11, k


def test_gated_norm_behind_the_gated_delta_rule():
    """The forward of the package's own recurrence, normed and gated by heads, and the
    gradient handed to its backward's dO: shapes, types and places fit without a copy."""
    B, T, Hh, K, V = 1, 128, 2, 64, 64
    q, k = (torch.nn.functional.normalize(rnd(B, T, Hh, K, seed=i), dim=-1).to(BF) for i in (1, 2))
    v, z = rnd(B, T, Hh, V, seed=3, dtype=BF), rnd(B, T, Hh, V, seed=4, dtype=BF)
    beta, g = torch.sigmoid(rnd(B, T, Hh, seed=5)), torch.nn.functional.logsigmoid(rnd(B, T, Hh, seed=6) + 2)
    o, _ = gdn.forward(q, k, v, beta, g, 64)
    w = rnd(V, seed=7, dtype=BF) + 1
    y = gdn.gate_norm_forward(o, z, w)
    f = o.double()
    ref = f * (f.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w.double() * torch.nn.functional.silu(z.double())
    # half a step of bf16, and 2^-18 of the values
    assert ((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -120).all()
    do, dz, dw, _ = gdn.gate_norm_backward(rnd(B, T, Hh, V, seed=8, dtype=BF), o, z, w)
    assert do.shape == o.shape and do.dtype == o.dtype and do.is_contiguous() and dz.shape == z.shape and dw.shape == (V,)


def test_two_streams_at_once():
    """The same calls on two streams at a time, each with workspaces of its own."""
    w = weights(BF)
    xs = [rnd(1, 3000, DM, seed=30 + i, dtype=BF) for i in range(2)]
    res = rnd(1, 3000, DM, seed=40, dtype=BF)

    def work(x):
        y, s, _ = gdn.layer_norm_forward(x, w["norm"], w["nbias"], res)
        z = torch.cat([y, y], -1)[..., :2 * P].contiguous()
        h, hT = gdn.glr_forward(z[..., :P], z[..., P:], form="sigmoid", scale="complement")
        grads = gdn.glr_backward(h, z[..., :P], z[..., P:], form="sigmoid", scale="complement")
        o = gdn.gate_norm_forward(heads(h) if h.shape[-1] == D else h, z[..., P:], w["gnorm"][0])
        return [y, s, h, hT, grads[0], grads[1], o, *gdn.layer_norm_backward(y, s, w["norm"], w["nbias"])]

    want = [work(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for st, x in zip(streams, xs):
            with torch.cuda.stream(st):
                got.append(work(x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))
