"""The layer operators run together, as a layer uses them: norm with the
residual's addition, projection, convolution, scan, projection; prompts in one
call, in two, and token by token from the pools; and a training step through
all of them against 64-bit autograd of the same formulas."""
import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DM, H, P, N, G, W = 96, 2, 64, 64, 1, 4
DC = H * P + 2 * G * N


def rnd(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def weights(dtype):
    return dict(norm=(1 + rnd(DM, seed=1, scale=0.1)).to(dtype), w_in=rnd(DM, DC + H, seed=2, dtype=dtype, scale=DM ** -0.5),
                conv=rnd(DC, W, seed=3, dtype=dtype, scale=0.5), cbias=rnd(DC, seed=4, dtype=dtype, scale=0.1),
                A=-torch.tensor([1.0, 4.0], device=DEV), D=rnd(H, seed=5), bias=torch.tensor([-3.0, -2.0], device=DEV),
                w_out=rnd(H * P, DM, seed=6, dtype=dtype, scale=(H * P) ** -0.5))


def parts(c):
    x, B, C = c.split((H * P, G * N, G * N), -1)
    return x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N))


def prompt(w, x, res, cstate=None, hstate=None, cu=None):
    y, s, _ = gdn.norm_forward(x, w["norm"], res)
    z = y @ w["w_in"]
    c, cs = gdn.conv_forward(z[..., :DC], w["conv"], w["cbias"], initial_state=cstate, cu_seqlens=cu)
    xs, B, C = parts(c)
    o, hs = gdn.ssm_forward(xs, z[..., DC:], w["A"], B, C, w["D"], w["bias"], hstate, cu_seqlens=cu)
    return o.flatten(2) @ w["w_out"], s, cs, hs


def token(w, x, res, cpool, hpool, slots):
    y, s, _ = gdn.norm_forward(x, w["norm"], res)
    z = y @ w["w_in"]
    c = gdn.conv_step(z[..., :DC], cpool, w["conv"], w["cbias"], slots=slots)
    xs, B, C = parts(c)
    o = gdn.ssm_step(xs, z[..., DC:], w["A"], B, C, hpool, w["D"], w["bias"], slots=slots)
    return o.flatten(1) @ w["w_out"], s


def test_prompt_then_tokens_is_one_prompt():
    """fp32: the same numbers by three ways.  Each value is a sum of at most a few
    hundred products in fp32, in another order each way: 2^-13 of the largest."""
    w, lens = weights(F32), [40, 130, 7]
    x, res = rnd(1, sum(lens), DM, seed=10), rnd(1, sum(lens), DM, seed=11)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    o, s, cs, hs = prompt(w, x, res, cu=cu)
    tol = float(o.abs().max()) * 2.0 ** -13
    # the first tokens of each as one packed prompt, the last five one by one
    k = 5
    heads = [n - k for n in lens]
    rows = torch.cat([torch.arange(n - k) + int(b) for n, b in zip(lens, cu[:-1])]).to(DEV)
    cu2 = torch.tensor([0] + heads).cumsum(0).to(torch.int32).to(DEV)
    o2, _, cs2, hs2 = prompt(w, x[:, rows].contiguous(), res[:, rows].contiguous(), cu=cu2)
    assert (o[:, rows] - o2).abs().max() <= tol
    cpool, hpool = rnd(6, W - 1, DC, seed=12), rnd(6, H, N, P, seed=13)
    slots = torch.tensor([4, 1, 5, -1], device=DEV, dtype=torch.int32)       # the last row is padding
    cpool[slots[:3].long()], hpool[slots[:3].long()] = cs2, hs2
    for t in range(k):
        at = torch.tensor([int(b) + n - k + t for n, b in zip(lens, cu[:-1])], device=DEV)
        xt = torch.cat([x[0, at], x[0, :1]])
        rt = torch.cat([res[0, at], res[0, :1]])
        ot, st = token(w, xt, rt, cpool, hpool, slots)
        assert (ot[:3] - o[0, at]).abs().max() <= tol, t
        assert torch.equal(st[:3], s[0, at])
    assert (cpool[slots[:3].long()] - cs).abs().max() <= float(cs.abs().max()) * 2.0 ** -13
    assert (hpool[slots[:3].long()] - hs).abs().max() <= float(hs.abs().max()) * 2.0 ** -13


def plain(w, x, res):
    """The layer's formulas in 64 bits, token by token."""
    s = x + res
    z = (s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w["norm"]) @ w["w_in"]
    pad = torch.cat([torch.zeros_like(z[:, :W - 1, :DC]), z[..., :DC]], 1)
    v = sum(w["conv"][:, j] * pad[:, j:j + z.shape[1]] for j in range(W)) + w["cbias"]
    xs, B, C = parts(v * torch.sigmoid(v))
    dt = torch.nn.functional.softplus(z[..., DC:] + w["bias"])
    h, out = torch.zeros(x.shape[0], H, N, P, dtype=x.dtype), []
    Bh, Ch = B.repeat_interleave(H // G, 2), C.repeat_interleave(H // G, 2)
    for t in range(x.shape[1]):
        h = torch.exp(dt[:, t] * w["A"])[..., None, None] * h + Bh[:, t][..., None] * (dt[:, t][..., None] * xs[:, t])[..., None, :]
        out.append((h * Ch[:, t][..., None]).sum(-2) + w["D"][:, None] * xs[:, t])
    return torch.stack(out, 1).flatten(2) @ w["w_out"], s


def test_training_step_through_the_layer():
    """fp32: gradients of all weights and inputs against 64-bit autograd.  Each way
    through the layer is a few hundred fp32 roundings of sums of both signs: each
    gradient within 2^-11 of its own norm."""
    w = weights(F32)
    B, T = 2, 90
    x, res, do, ds = (rnd(B, T, DM, seed=20 + i) for i in range(4))
    y, s, _ = gdn.norm_forward(x, w["norm"], res)
    z = y @ w["w_in"]
    c, _ = gdn.conv_forward(z[..., :DC], w["conv"], w["cbias"])
    xs, Bm, Cm = parts(c)
    o, _ = gdn.ssm_forward(xs, z[..., DC:], w["A"], Bm, Cm, w["D"], w["bias"])
    got = {"w_out": o.flatten(0, 1).flatten(1).T @ do.flatten(0, 1)}
    dy = (do @ w["w_out"].T).unflatten(-1, (H, P))
    # the scan's gradients go straight into the buffer that the convolution reads
    dc = torch.empty(B, T, DC, device=DEV)
    dxs, dB, dC = parts(dc)
    _, ddt, got["A"], _, _, got["D"], got["bias"], _ = gdn.ssm_backward(dy, xs, z[..., DC:], w["A"], Bm, Cm, w["D"], w["bias"],
                                                                         dx=dxs, dB=dB, dC=dC)
    dz, got["conv"], got["cbias"], _ = gdn.conv_backward(dc, z[..., :DC], w["conv"], w["cbias"])
    dz = torch.cat([dz, ddt], -1)
    got["w_in"] = y.flatten(0, 1).T @ dz.flatten(0, 1)
    got["x"], _, got["norm"] = gdn.norm_backward(dz @ w["w_in"].T, s, w["norm"], ds)
    leaves = {k: v.detach().cpu().double().requires_grad_() for k, v in {**w, "x": x}.items()}
    out, kept = plain(leaves, leaves["x"], res.cpu().double())
    ((out * do.cpu().double()).sum() + (kept * ds.cpu().double()).sum()).backward()
    for k, v in got.items():
        ref = leaves[k].grad
        assert (v.cpu().double() - ref).norm() <= ref.norm() * 2.0 ** -11, k


def test_eight_bit_rows_feed_a_product():
    """A norm's e4m3 rows and scales stand for its rows: within half a step, 2^-4."""
    w = weights(BF)
    x, res = rnd(70, DM, seed=10, dtype=BF), rnd(70, DM, seed=11, dtype=BF)
    y, s, _ = gdn.norm_forward(x, w["norm"], res)
    q, s8, scale = gdn.norm_forward(x, w["norm"], res, out_dtype=torch.float8_e4m3fn)
    assert torch.equal(s, s8)
    back = q.float() * scale
    assert ((back - y.float()).abs() <= y.float().abs() * (2.0 ** -4 + 2.0 ** -8) + scale * 2.0 ** -10).all()
