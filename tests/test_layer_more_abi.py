"""Host-only checks of layer norm's, the gated norm's and the gated linear
recurrence's C ABI and binding: bad arguments are refused before any GPU work is
enqueued (every call below returns during validation, or has nothing to do)."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer as L

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 6
P = ctypes.c_void_p
FAKE, ODD8, ODD2, ODD1 = P(0x10000), P(0x10008), P(0x10002), P(0x10001)     # never dereferenced
BIG = ctypes.c_size_t(1 << 50)
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from chunked_gated_delta_prepare_amd import build
        build.build()
    return gdn.load_library()


def test_package_reaches_every_operator():
    for name in ("layer_norm_forward", "layer_norm_backward", "gate_norm_forward", "gate_norm_backward", "glr_forward",
                 "glr_backward", "glr_step"):
        assert getattr(gdn, name) is getattr(L, name) and name in gdn.__all__


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def ln_problem(**kw):
    d = dict(rows=5, D=64, x_stride=64, x_dtype=1, s_dtype=1, w_dtype=1, out_dtype=1, group=0, eps=1e-6)
    d.update(kw)
    return L.NormProblem(**d)


def ln_forward(lib, pr, x=FAKE, residual=FAKE, w=FAKE, b=FAKE, y=FAKE, s=FAKE, scales=FAKE):
    return lib.gdn_layer_norm_forward(ctypes.byref(pr), x, residual, w, b, y, s, scales, None)


def ln_backward(lib, pr, dy=FAKE, s=FAKE, w=FAKE, dres=FAKE, ds=FAKE, dx=None, dw=FAKE, db=FAKE, ws=FAKE, size=BIG):
    return lib.gdn_layer_norm_backward(ctypes.byref(pr), dy, s, w, dres, ds, dx, dw, db, ws, size, None)


@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, SHAPE), ("D", 0, SHAPE), ("eps", -1.0, SHAPE), ("eps", float("nan"), SHAPE), ("D", 16385, UNSUPPORTED),
    ("rows", 1 << 31, UNSUPPORTED), ("x_dtype", 2, UNSUPPORTED), ("s_dtype", 3, UNSUPPORTED), ("w_dtype", 2, UNSUPPORTED),
    ("out_dtype", 0, UNSUPPORTED), ("group", 64, UNSUPPORTED)])
def test_layer_norm_problems_refused(lib, field, value, status):
    pr = ln_problem(**{field: value})
    assert ln_forward(lib, pr) == status and ln_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_layer_norm_backward(ctypes.byref(pr)) == 0


def test_layer_norm_arguments(lib):
    pr = ln_problem()
    assert lib.gdn_layer_norm_forward(None, FAKE, None, FAKE, None, FAKE, None, None, None) == NULL
    for k in ("x", "w", "y", "s"):
        assert ln_forward(lib, pr, **{k: None}) == NULL, k
    assert ln_forward(lib, ln_problem(out_dtype=2), scales=None) == NULL
    assert ln_forward(lib, ln_problem(s_dtype=0), residual=None) == UNSUPPORTED
    for k in ("x", "w", "b", "y", "s", "residual"):
        assert ln_forward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert ln_forward(lib, ln_problem(out_dtype=2), scales=ODD2) == ALIGN
    assert ln_forward(lib, ln_problem(rows=0), x=None, residual=None, w=None, b=None, y=None, s=None, scales=None) == OK
    for k in ("dy", "s", "w", "ds", "dw"):
        assert ln_backward(lib, pr, **{k: None}) == NULL, k
    for k in ("dy", "s", "w", "dres", "ds", "dx", "dw", "db"):
        assert ln_backward(lib, pr, **{k: ODD1}) == ALIGN, k
    need = lib.gdn_workspace_bytes_layer_norm_backward(ctypes.byref(pr))
    assert need == 2 * 8 * 64 * 4            # two workgroups of four rows, of dw and db
    assert ln_backward(lib, pr, ws=None, size=0) == WORKSPACE and ln_backward(lib, pr, size=need - 1) == WORKSPACE
    assert ln_backward(lib, pr, ws=ODD8) == ALIGN
    # the workgroups share the rows evenly: 1003 rows two at a time
    assert lib.gdn_workspace_bytes_layer_norm_backward(ctypes.byref(ln_problem(rows=1003, D=2050))) == 502 * 2050 * 8


# ---------------------------------------------------------------------------
# gated norm
# ---------------------------------------------------------------------------

def gn_problem(**kw):
    d = dict(T=6, H=4, D=64, x_stride_t=256, x_stride_h=64, z_stride_t=512, z_stride_h=64, dz_stride_t=512, dz_stride_h=64,
             io_dtype=1, w_dtype=1, each=0, gate_first=0, center=1, act=0, eps=1e-6)
    d.update(kw)
    return L.GateNormProblem(**d)


def gn_forward(lib, pr, x=FAKE, z=FAKE, w=FAKE, b=FAKE, y=FAKE):
    return lib.gdn_gate_norm_forward(ctypes.byref(pr), x, z, w, b, y, None)


def gn_backward(lib, pr, dy=FAKE, x=FAKE, z=FAKE, w=FAKE, b=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, db=FAKE, ws=FAKE, size=BIG):
    return lib.gdn_gate_norm_backward(ctypes.byref(pr), dy, x, z, w, b, dx, dz, dw, db, ws, size, None)


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, SHAPE), ("H", 0, SHAPE), ("D", 0, SHAPE), ("eps", -1.0, SHAPE), ("eps", float("nan"), SHAPE), ("D", 8193, UNSUPPORTED),
    ("T", 1 << 30, UNSUPPORTED), ("H", 1 << 31, UNSUPPORTED), ("io_dtype", 2, UNSUPPORTED), ("w_dtype", 2, UNSUPPORTED), ("act", 2, UNSUPPORTED)])
def test_gate_norm_problems_refused(lib, field, value, status):
    pr = gn_problem(**{field: value})
    assert gn_forward(lib, pr) == status and gn_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_gate_norm_backward(ctypes.byref(pr)) == 0


def test_gate_norm_arguments(lib):
    pr = gn_problem()
    assert lib.gdn_gate_norm_forward(None, FAKE, FAKE, FAKE, None, FAKE, None) == NULL
    for k in ("x", "z", "w", "y"):
        assert gn_forward(lib, pr, **{k: None}) == NULL, k
    for k in ("x", "z", "w", "b", "y"):
        assert gn_forward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert gn_forward(lib, gn_problem(center=0)) == UNSUPPORTED              # a bias without a mean
    assert gn_forward(lib, gn_problem(each=1, H=65537)) == UNSUPPORTED
    assert gn_forward(lib, gn_problem(T=0), x=None, z=None, w=None, b=None, y=None) == OK
    for k in ("dy", "x", "z", "w", "dx", "dz", "dw"):
        assert gn_backward(lib, pr, **{k: None}) == NULL, k
    for k in ("dy", "x", "z", "w", "b", "dx", "dz", "dw", "db"):
        assert gn_backward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert gn_backward(lib, gn_problem(center=0), b=None) == UNSUPPORTED     # nor a bias's gradient
    need = lib.gdn_workspace_bytes_gate_norm_backward(ctypes.byref(pr))
    assert need == 2 * 64 * 4                # 24 rows in one workgroup of 16 slots, two rows each
    assert lib.gdn_workspace_bytes_gate_norm_backward(ctypes.byref(gn_problem(each=1))) == 4 * 2 * 64 * 4      # one for each head
    assert gn_backward(lib, pr, ws=None, size=0) == WORKSPACE and gn_backward(lib, pr, size=need - 1) == WORKSPACE
    assert gn_backward(lib, pr, ws=ODD8) == ALIGN


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------

def glr_problem(**kw):
    d = dict(B=2, T=100, D=64, n_seqs=0, io_dtype=1, g_dtype=1, form=2, scale=2)
    for k in ("x", "g", "dy", "dx", "dg"):
        d[k + "_stride_b"], d[k + "_stride_t"] = 6400, 64
    d.update(kw)
    return L.GlrProblem(**d)


def glr_forward(lib, pr, x=FAKE, gate=FAKE, bias=FAKE, rate=FAKE, h0=FAKE, cu=None, y=FAKE, hT=FAKE, ws=FAKE, size=BIG):
    return lib.gdn_glr_forward(ctypes.byref(pr), x, gate, bias, rate, h0, cu, y, hT, ws, size, None)


def glr_backward(lib, pr, **kw):
    names = ("dy", "x", "gate", "bias", "rate", "h0", "cu", "dhT", "dx", "dgate", "dbias", "drate", "dh0", "ws")
    a = [kw.get(n, None if n == "cu" else FAKE) for n in names]
    return lib.gdn_glr_backward(ctypes.byref(pr), *a, kw.get("size", BIG), None)


def glr_step(lib, pr, x=FAKE, gate=FAKE, bias=FAKE, rate=FAKE, state=FAKE, slots=FAKE, n=8, y=FAKE):
    return lib.gdn_glr_step(ctypes.byref(pr), x, gate, bias, rate, state, slots, n, y, None)


@pytest.mark.parametrize("field,value,status", [
    ("B", 0, SHAPE), ("T", -1, SHAPE), ("D", 0, SHAPE), ("io_dtype", 2, UNSUPPORTED), ("g_dtype", 2, UNSUPPORTED), ("form", 3, UNSUPPORTED),
    ("form", -1, UNSUPPORTED), ("scale", 3, UNSUPPORTED), ("T", (1 << 30) + 1, UNSUPPORTED), ("D", (1 << 20) + 1, UNSUPPORTED),
    ("B", 1 << 24, UNSUPPORTED), ("x_stride_t", -64, UNSUPPORTED), ("g_stride_t", (1 << 20) + 1, UNSUPPORTED),
    ("dg_stride_t", (1 << 20) + 1, UNSUPPORTED)])
def test_glr_problems_refused(lib, field, value, status):
    pr = glr_problem(**{field: value})
    assert glr_forward(lib, pr) == status and glr_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_glr(ctypes.byref(pr)) == 0 and lib.gdn_workspace_bytes_glr_backward(ctypes.byref(pr)) == 0
    assert glr_step(lib, glr_problem(**{"T": 1, field: value})) in (status, SHAPE)


def test_glr_arguments(lib):
    pr = glr_problem()
    assert lib.gdn_glr_forward(None, *[FAKE] * 9, BIG, None) == NULL
    for k in ("x", "gate", "y", "rate"):
        assert glr_forward(lib, pr, **{k: None}) == NULL, k
    for k in ("x", "gate", "bias", "rate", "h0", "y", "hT"):
        assert glr_forward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert glr_forward(lib, glr_problem(form=0)) == UNSUPPORTED              # a rate without its form
    assert glr_forward(lib, glr_problem(n_seqs=3), cu=FAKE) == SHAPE         # packed means B = 1
    assert glr_forward(lib, glr_problem(B=1), cu=FAKE) == SHAPE
    assert glr_forward(lib, glr_problem(B=1, n_seqs=3), cu=ODD2) == ALIGN
    assert glr_forward(lib, glr_problem(T=0), x=None, gate=None, y=None, hT=None) == OK
    for k in ("dy", "x", "gate", "dx", "dgate", "rate"):
        assert glr_backward(lib, pr, **{k: None}) == NULL, k
    for k in ("dy", "x", "gate", "bias", "rate", "h0", "dhT", "dx", "dgate", "dbias", "drate", "dh0"):
        assert glr_backward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert glr_backward(lib, glr_problem(form=0), rate=None) == UNSUPPORTED  # nor a rate's gradient
    need = lib.gdn_workspace_bytes_glr_backward(ctypes.byref(pr))
    assert need == 2 * 4 * 5 * 64 * 4        # four tiles of 32 tokens a sequence: three numbers and two sums a channel
    assert glr_backward(lib, pr, size=need - 1) == WORKSPACE and glr_backward(lib, pr, ws=None, size=0) == WORKSPACE
    assert glr_backward(lib, pr, ws=ODD8) == ALIGN
    assert lib.gdn_workspace_bytes_glr(ctypes.byref(pr)) == 0                # one segment
    many = glr_problem(B=1, T=5000)
    need = lib.gdn_workspace_bytes_glr(ctypes.byref(many))
    assert need > 0 and glr_forward(lib, many, size=need - 1) == WORKSPACE and glr_forward(lib, many, ws=ODD8) == ALIGN
    one = glr_problem(T=1)
    assert glr_step(lib, pr) == SHAPE and glr_step(lib, one, n=-1) == SHAPE and glr_step(lib, one, slots=None, n=1) == SHAPE
    for k in ("x", "gate", "rate", "state", "y"):
        assert glr_step(lib, one, **{k: None}) == NULL, k
    assert glr_step(lib, one, slots=ODD2) == ALIGN and glr_step(lib, one, state=ODD2) == ALIGN


# ---------------------------------------------------------------------------
# the binding: calls are caught at the library's door, with CPU tensors
# ---------------------------------------------------------------------------

@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(L, "_device", lambda t, name: t.device)
    monkeypatch.setattr(L, "_on", lambda device, stream, work, *args: work(None, *args))
    monkeypatch.setattr(L, "_call", lambda name, pr, *args: seen.append((name, pr._obj, args)))
    return seen


def test_gate_norm_strides(calls):
    T, H, D = 6, 4, 64
    x, w = torch.zeros(T, H, D), torch.ones(D)
    z = torch.zeros(T, 700)[:, 100:100 + H * D].unflatten(-1, (H, D))
    gdn.gate_norm_forward(x, z, w)
    heads_first = torch.zeros(H, T, D).transpose(0, 1)
    gdn.gate_norm_forward(heads_first, z, torch.ones(H, D))
    gdn.gate_norm_forward(x.unflatten(0, (2, 3)), z.unflatten(0, (2, 3)), w)
    gdn.gate_norm_forward(x[:, 0], z[:, 0], w)
    pr = [c[1] for c in calls]
    assert [(p.T, p.H, p.x_stride_t, p.x_stride_h, p.z_stride_t, p.z_stride_h, p.each) for p in pr] == [
        (T, H, H * D, D, 700, D, 0), (T, H, D, T * D, 700, D, 1), (T, H, H * D, D, 700, D, 0), (T, 1, H * D, D, 700, D, 0)]
    with pytest.raises(ValueError, match="one stride"):
        gdn.gate_norm_forward(torch.zeros(2, 4, H, D)[:, :3], z.unflatten(0, (2, 3)), w)
    for dz in (torch.zeros(1, H, D).expand(T, H, D), torch.zeros(T, 1, D).expand(T, H, D), torch.zeros(T * 100).as_strided((T, H, D), (80, 20, 1))):
        with pytest.raises(ValueError, match="overlap"):
            gdn.gate_norm_backward(x, x, z, w, dz=dz)
    ok = torch.zeros(H, T, D).transpose(0, 1)
    assert gdn.gate_norm_backward(x, x, z, w, dz=ok)[1] is ok


def test_glr_gradients_side_by_side(calls):
    B, T, D = 2, 7, 64
    x, gate = torch.zeros(B, T, D), torch.zeros(B, T, D)
    dx, dg, *_ = gdn.glr_backward(x, x, gate)
    assert dx.is_contiguous() and dg.is_contiguous()
    buf = torch.zeros(B, T, 2 * D + 5)
    gdn.glr_backward(x, x, gate, dx=buf[..., D:2 * D], dgate=buf[..., :D])
    gdn.glr_backward(x, x, gate, dx=torch.zeros(B, T, D), dgate=torch.zeros(B, T, D))
    gdn.glr_backward(x, x, gate, dx=torch.zeros(B, T, D))
    assert len(calls) == 4
    for one, two in ((buf[..., :D], buf[..., D - 1:2 * D - 1]), (buf[..., :D], buf[..., :D]), (buf[..., 5:5 + D], torch.zeros(B, 1, D).expand(B, T, D)),
                     (torch.zeros(B * T * 40 + D).as_strided((B, T, D), (T * 40, 40, 1)), None)):
        with pytest.raises(ValueError, match="overlap|share"):
            gdn.glr_backward(x, x, gate, dx=one, dgate=two)
    with pytest.raises(ValueError, match="share"):
        gdn.glr_backward(x, x, gate, dx=x)


def test_states_share_memory_with_no_input(calls):
    B, D, S = 3, 64, 5
    pool = torch.zeros(S, D)
    d = dict(x=torch.zeros(B, D), gate=torch.zeros(B, D), gate_bias=torch.zeros(D), rate=torch.ones(D), slots=torch.zeros(B, dtype=torch.int32))
    gdn.glr_step(**d, state=pool, form="rate")
    for k in d:
        inside = (pool.view(torch.int32) if k == "slots" else pool).view(-1)[64:64 + d[k].numel()].view(d[k].shape)
        with pytest.raises(ValueError, match="share memory"):
            gdn.glr_step(**{**d, k: inside}, state=pool, form="rate")
    with pytest.raises(ValueError, match="share memory"):
        gdn.glr_step(**{**d, "x": pool.as_strided((B, D), (2, 1))}, state=pool, form="rate")


def test_outputs_that_would_not_be_written_are_refused(calls):
    x, w = torch.zeros(4, 64), torch.ones(64)
    for bad, name in ((lambda: gdn.layer_norm_forward(x, w, s=torch.zeros(4, 64)), "residual"),
                      (lambda: gdn.layer_norm_forward(x, w, scales=torch.zeros(4, 1)), "scales"),
                      (lambda: gdn.layer_norm_backward(x, x, w, dbias=torch.zeros(64)), "dbias"),
                      (lambda: gdn.gate_norm_backward(x, x, x, w, dbias=torch.zeros(64)), "dbias"),
                      (lambda: gdn.glr_backward(x[None], x[None], x[None], dbias=torch.zeros(64)), "dbias"),
                      (lambda: gdn.glr_backward(x[None], x[None], x[None], drate=torch.zeros(64)), "drate"),
                      (lambda: gdn.glr_backward(x[None], x[None], x[None], dh0=torch.zeros(1, 64)), "dh0")):
        with pytest.raises(ValueError, match=name):
            bad()
    assert not calls
