"""Host-only checks of the layer operators' C ABI (include/libgdn_layer.h) and
binding: everything declared is exported, and bad arguments are refused before
any GPU work is enqueued (every call below returns during validation)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 6
P = ctypes.c_void_p
FAKE, ODD8, ODD2, ODD1 = P(0x10000), P(0x10008), P(0x10002), P(0x10001)     # never dereferenced
BIG = ctypes.c_size_t(1 << 50)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from chunked_gated_delta_prepare_amd import build
        build.build()
    return gdn.load_library()


def _declared():
    src = open(os.path.join(ROOT, "include", "libgdn_layer.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*[A-Za-z_][\w \*]*?\b(gdn_\w+)\s*\(", src, flags=re.M)))


def test_header_binding_and_library_agree(lib):
    assert _declared() == sorted(L.LAYER_EXPORTS)
    for name in _declared():
        assert hasattr(lib, name), name
    if os.path.exists(gdn.POISON_LIB_PATH):
        dbg = gdn.load_library(gdn.POISON_LIB_PATH)
        for name in _declared():
            assert hasattr(dbg, name), name


def test_package_reaches_every_operator():
    for name in ("norm_forward", "norm_backward", "conv_forward", "conv_backward", "conv_step", "ssm_forward",
                 "ssm_backward", "ssm_step"):
        assert getattr(gdn, name) is getattr(L, name) and name in gdn.__all__
    with pytest.raises(AttributeError):
        gdn.no_such_operator


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def norm_problem(**kw):
    d = dict(rows=5, D=64, x_stride=64, x_dtype=1, s_dtype=1, w_dtype=1, out_dtype=1, group=0, eps=1e-6)
    d.update(kw)
    return L.NormProblem(**d)


def norm_forward(lib, pr, x=FAKE, residual=FAKE, w=FAKE, y=FAKE, s=FAKE, scales=FAKE):
    return lib.gdn_norm_forward(ctypes.byref(pr), x, residual, w, y, s, scales, None)


def norm_backward(lib, pr, dy=FAKE, s=FAKE, w=FAKE, dres=FAKE, ds=FAKE, dx=None, dw=FAKE, ws=FAKE, size=BIG):
    return lib.gdn_norm_backward(ctypes.byref(pr), dy, s, w, dres, ds, dx, dw, ws, size, None)


@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, SHAPE), ("D", 0, SHAPE), ("eps", -1.0, SHAPE), ("eps", float("nan"), SHAPE), ("D", 16385, UNSUPPORTED),
    ("rows", 1 << 31, UNSUPPORTED), ("x_dtype", 2, UNSUPPORTED), ("s_dtype", 3, UNSUPPORTED), ("w_dtype", 2, UNSUPPORTED),
    ("out_dtype", 0, UNSUPPORTED), ("group", 64, UNSUPPORTED)])
def test_norm_problems_refused(lib, field, value, status):
    pr = norm_problem(**{field: value})
    assert norm_forward(lib, pr) == status
    assert norm_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_norm_backward(ctypes.byref(pr)) == 0


def test_norm_arguments(lib):
    pr = norm_problem()
    assert lib.gdn_norm_forward(None, FAKE, None, FAKE, FAKE, None, None, None) == NULL
    for k in ("x", "w", "y", "s"):
        assert norm_forward(lib, pr, **{k: None}) == NULL, k
    assert norm_forward(lib, norm_problem(out_dtype=2), scales=None) == NULL
    assert norm_forward(lib, norm_problem(s_dtype=0), residual=None) == UNSUPPORTED      # s would be x, in x's type
    for k in ("x", "w", "y", "s", "residual"):
        assert norm_forward(lib, pr, **{k: ODD1}) == ALIGN, k
    assert norm_forward(lib, norm_problem(out_dtype=2), scales=ODD2) == ALIGN
    assert norm_forward(lib, norm_problem(rows=0), x=None, residual=None, w=None, y=None, s=None, scales=None) == OK
    for k in ("dy", "s", "w", "ds", "dw"):
        assert norm_backward(lib, pr, **{k: None}) == NULL, k
    for k in ("dy", "s", "w", "dres", "ds", "dx", "dw"):
        assert norm_backward(lib, pr, **{k: ODD1}) == ALIGN, k
    need = lib.gdn_workspace_bytes_norm_backward(ctypes.byref(pr))
    assert need == 8 * 64 * 4            # two workgroups of four rows
    assert norm_backward(lib, pr, ws=None, size=0) == WORKSPACE
    assert norm_backward(lib, pr, size=need - 1) == WORKSPACE
    assert norm_backward(lib, pr, ws=ODD8) == ALIGN


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def conv_problem(**kw):
    d = dict(B=2, T=100, D=64, W=4, x_stride_b=6400, x_stride_t=64, dy_stride_b=6400, dy_stride_t=64, n_seqs=0,
             io_dtype=1, w_dtype=1, silu=1)
    d.update(kw)
    return L.ConvProblem(**d)


def conv_forward(lib, pr, x=FAKE, w=FAKE, b=FAKE, init=None, cu=None, y=FAKE, final=FAKE):
    return lib.gdn_conv_forward(ctypes.byref(pr), x, w, b, init, cu, y, final, None)


def conv_backward(lib, pr, dy=FAKE, x=FAKE, w=FAKE, b=FAKE, init=None, cu=None, df=None, dx=FAKE, dw=FAKE, db=FAKE, di=None,
                  ws=FAKE, size=BIG):
    return lib.gdn_conv_backward(ctypes.byref(pr), dy, x, w, b, init, cu, df, dx, dw, db, di, ws, size, None)


def conv_step(lib, pr, x=FAKE, w=FAKE, b=FAKE, state=FAKE, slots=FAKE, n=8, y=FAKE):
    return lib.gdn_conv_step(ctypes.byref(pr), x, w, b, state, slots, n, y, None)


@pytest.mark.parametrize("field,value,status", [
    ("B", 0, SHAPE), ("T", -1, SHAPE), ("D", 0, SHAPE), ("W", 0, SHAPE), ("W", 1, UNSUPPORTED), ("W", 5, UNSUPPORTED),
    ("io_dtype", 2, UNSUPPORTED), ("w_dtype", 2, UNSUPPORTED), ("x_stride_t", -64, UNSUPPORTED),
    ("x_stride_t", (1 << 23) + 1, UNSUPPORTED), ("D", (1 << 23) + 1, UNSUPPORTED), ("T", (1 << 30) + 1, UNSUPPORTED),
    ("B", (1 << 24) + 1, UNSUPPORTED)])
def test_conv_problems_refused(lib, field, value, status):
    pr = conv_problem(**{field: value})
    assert conv_forward(lib, pr) == status
    assert conv_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_conv_backward(ctypes.byref(pr)) == 0
    one = conv_problem(**{"T": 1, field: value})
    assert conv_step(lib, one) in (status, SHAPE)


def test_conv_arguments(lib):
    pr = conv_problem()
    assert lib.gdn_conv_forward(None, FAKE, FAKE, None, None, None, FAKE, None, None) == NULL
    for k in ("x", "w", "y"):
        assert conv_forward(lib, pr, **{k: None}) == NULL, k
    for k in ("x", "w", "b", "init", "y", "final"):
        assert conv_forward(lib, pr, **{k: ODD1}) == ALIGN, k
    packed = conv_problem(B=1, n_seqs=3)
    assert conv_forward(lib, packed, cu=ODD2) == ALIGN
    assert conv_forward(lib, conv_problem(B=2, n_seqs=3), cu=FAKE) == SHAPE        # packed means B = 1
    assert conv_forward(lib, conv_problem(B=1, n_seqs=0), cu=FAKE) == SHAPE
    for k in ("dy", "x", "w", "dx", "dw"):
        assert conv_backward(lib, pr, **{k: None}) == NULL, k
    need = lib.gdn_workspace_bytes_conv_backward(ctypes.byref(pr))
    assert need == 2 * 5 * 64 * 4        # eight runs of 32 tokens, four a workgroup
    assert conv_backward(lib, pr, size=need - 1) == WORKSPACE
    assert conv_backward(lib, pr, ws=None, size=0) == WORKSPACE
    assert conv_backward(lib, pr, ws=ODD8) == ALIGN
    one = conv_problem(T=1)
    assert conv_step(lib, pr) == SHAPE                                               # T must be 1
    assert conv_step(lib, one, n=-1) == SHAPE
    assert conv_step(lib, one, slots=None, n=1) == SHAPE                              # a state per row
    for k in ("x", "w", "state", "y"):
        assert conv_step(lib, one, **{k: None}) == NULL, k
    assert conv_step(lib, one, slots=ODD2) == ALIGN


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def ssm_problem(**kw):
    d = dict(B=2, T=1000, H=4, P=64, N=128, G=2, x_stride_b=1 << 20, x_stride_t=256, bc_stride_b=1 << 20, bc_stride_t=256,
             dt_stride_b=4000, dt_stride_t=4, dxbc_stride_b=1 << 20, dxbc_stride_t=256, n_seqs=0, io_dtype=1, dt_dtype=1,
             softplus=1)
    d.update(kw)
    return L.SsmProblem(**d)


def ssm_forward(lib, pr, x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, D=FAKE, bias=FAKE, h0=None, cu=None, y=FAKE, hT=FAKE,
                ws=FAKE, size=BIG):
    return lib.gdn_ssm_forward(ctypes.byref(pr), x, dt, A, B, C, D, bias, h0, cu, y, hT, ws, size, None)


def ssm_backward(lib, pr, **kw):
    names = ("dy", "x", "dt", "A", "B", "C", "D", "bias", "h0", "cu", "dhT", "dx", "ddt", "dA", "dB", "dC", "dD", "dbias",
             "dh0", "ws")
    a = [kw.get(n, None if n in ("h0", "cu", "dhT", "dh0") else FAKE) for n in names]
    return lib.gdn_ssm_backward(ctypes.byref(pr), *a, kw.get("size", BIG), None)


def ssm_step(lib, pr, x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, D=FAKE, bias=FAKE, state=FAKE, slots=FAKE, n=8, y=FAKE):
    return lib.gdn_ssm_step(ctypes.byref(pr), x, dt, A, B, C, D, bias, state, slots, n, y, None)


@pytest.mark.parametrize("field,value,status", [
    ("B", 0, SHAPE), ("T", -1, SHAPE), ("H", 0, SHAPE), ("G", 0, SHAPE), ("G", 3, SHAPE), ("P", 0, SHAPE), ("N", 0, SHAPE),
    ("P", 96, UNSUPPORTED), ("N", 32, UNSUPPORTED), ("io_dtype", 2, UNSUPPORTED), ("dt_dtype", 2, UNSUPPORTED),
    ("x_stride_t", -8, UNSUPPORTED), ("bc_stride_t", (1 << 22) + 8, UNSUPPORTED), ("dt_stride_t", -1, UNSUPPORTED),
    ("dxbc_stride_t", -8, UNSUPPORTED), ("T", (1 << 30) + 1, UNSUPPORTED), ("B", (1 << 20) + 1, UNSUPPORTED)])
def test_ssm_problems_refused(lib, field, value, status):
    pr = ssm_problem(**{field: value})
    assert ssm_forward(lib, pr) == status
    assert ssm_backward(lib, pr) == status
    assert lib.gdn_workspace_bytes_ssm(ctypes.byref(pr)) == 0
    assert lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(pr)) == 0


def test_launches_of_too_many_threads_refused(lib):
    # 2^32 threads in a launch: runs of 32 tokens a wave; heads and their blocks a workgroup
    assert conv_forward(lib, conv_problem(B=2, T=1 << 30, D=1)) == UNSUPPORTED
    assert conv_step(lib, conv_problem(B=1 << 24, T=1, D=200), n=1 << 24) == UNSUPPORTED
    many = ssm_problem(B=1 << 20, T=1, H=64, G=1, x_stride_t=64 * 64, dxbc_stride_t=64 * 64)
    assert ssm_forward(lib, many) == UNSUPPORTED and ssm_backward(lib, many) == UNSUPPORTED
    assert ssm_step(lib, many, n=1 << 20) == UNSUPPORTED
    assert lib.gdn_workspace_bytes_ssm(ctypes.byref(many)) == 0
    # a problem under them has a workspace
    assert lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(ssm_problem(B=1 << 14, T=1, H=64, G=1, x_stride_t=64 * 64))) > 0


@pytest.mark.parametrize("B,T,D", [(1 << 24, ((1 << 24) - 1) * 32, 1 << 23), (1 << 24, ((1 << 25) - 1) * 32, 1 << 22),
                                   (1 << 22, ((1 << 22) - 1) * 32, 1 << 20)])
def test_launches_whose_size_passes_64_bits_refused(lib, B, T, D):
    pr = conv_problem(B=B, T=T, D=D, x_stride_b=0, x_stride_t=0, dy_stride_b=0, dy_stride_t=0)
    assert conv_forward(lib, pr) == UNSUPPORTED and conv_backward(lib, pr) == UNSUPPORTED
    assert lib.gdn_workspace_bytes_conv_backward(ctypes.byref(pr)) == 0


def test_ssm_overlapping_rows_refused(lib):
    # a token's row would reach into the next one's
    assert ssm_forward(lib, ssm_problem(x_stride_t=128)) == UNSUPPORTED
    assert ssm_forward(lib, ssm_problem(bc_stride_t=128)) == UNSUPPORTED
    assert ssm_backward(lib, ssm_problem(dxbc_stride_t=128)) == UNSUPPORTED


def test_ssm_arguments(lib):
    pr = ssm_problem()
    for k in ("x", "dt", "A", "B", "C", "y"):
        assert ssm_forward(lib, pr, **{k: None}) == NULL, k
    for k in ("x", "B", "C", "y", "ws"):
        assert ssm_forward(lib, pr, **{k: ODD8}) == ALIGN, k
    for k in ("A", "D", "bias", "h0", "hT"):
        assert ssm_forward(lib, pr, **{k: ODD2}) == ALIGN, k
    assert ssm_forward(lib, pr, dt=ODD1) == ALIGN
    assert ssm_forward(lib, ssm_problem(x_stride_t=257)) == ALIGN
    assert ssm_forward(lib, ssm_problem(B=1, n_seqs=2), cu=ODD2) == ALIGN
    assert ssm_forward(lib, ssm_problem(n_seqs=2), cu=FAKE) == SHAPE                  # packed means B = 1
    # 2 x 2 streams of 128 columns, 16 chunks in four segments of four
    need = lib.gdn_workspace_bytes_ssm(ctypes.byref(pr))
    assert need == 2 * 4 * 2 * (16 + 128 * 128 * 4)
    assert ssm_forward(lib, pr, ws=None, size=0) == WORKSPACE
    assert ssm_forward(lib, pr, size=need - 1) == WORKSPACE
    assert lib.gdn_workspace_bytes_ssm(ctypes.byref(ssm_problem(T=256))) == 0         # one segment
    assert lib.gdn_workspace_bytes_ssm(ctypes.byref(ssm_problem(T=0))) == 0
    assert ssm_forward(lib, ssm_problem(T=0), x=None, dt=None, A=None, B=None, C=None, y=None, hT=None, ws=None) == OK
    for k in ("dy", "x", "dt", "A", "B", "C", "dx", "ddt", "dA", "dB", "dC"):
        assert ssm_backward(lib, pr, **{k: None}) == NULL, k
    for k in ("dy", "dx", "dB", "dC", "ws"):
        assert ssm_backward(lib, pr, **{k: ODD8}) == ALIGN, k
    need = lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(pr))
    assert ssm_backward(lib, pr, size=need - 1) == WORKSPACE
    assert ssm_backward(lib, pr, ws=None, size=0) == WORKSPACE
    one = ssm_problem(T=1)
    assert ssm_step(lib, pr) == SHAPE
    assert ssm_step(lib, one, slots=None, n=1) == SHAPE
    for k in ("x", "dt", "A", "B", "C", "state", "y"):
        assert ssm_step(lib, one, **{k: None}) == NULL, k
    assert ssm_step(lib, one, state=ODD8) == ALIGN
    assert ssm_step(lib, one, slots=ODD2) == ALIGN


def test_ssm_gates_wanted_without_tokens(lib):
    # no token, but final states to write: the kernel reads A
    none = dict(x=None, dt=None, B=None, C=None, y=None, ws=None)
    for packed in (dict(), dict(B=1, n_seqs=2)):
        pr = ssm_problem(T=0, **packed)
        cu = FAKE if packed else None
        assert ssm_forward(lib, pr, A=None, cu=cu, **none) == NULL
        for k in ("A", "D", "bias"):
            assert ssm_forward(lib, pr, **{**none, k: ODD2}, cu=cu) == ALIGN, k
    assert ssm_forward(lib, ssm_problem(T=0), A=None, hT=None, **none) == OK


def packed_scan(T, n, H, P, N, G):
    return ssm_problem(B=1, T=T, n_seqs=n, H=H, P=P, N=N, G=G, x_stride_t=H * P, bc_stride_t=G * N, dt_stride_t=H,
                       dxbc_stride_t=H * P)


def test_many_short_packed_sequences_are_taken(lib):
    # the backward's launches follow the tokens, not sequences times segments
    for T, n in ((262144, 4096), (1 << 20, 1 << 14)):
        pr = packed_scan(T, n, 64, 128, 128, 8)
        assert ssm_forward(lib, pr, cu=FAKE, ws=None, size=0) == WORKSPACE
        assert ssm_backward(lib, pr, cu=FAKE, ws=None, size=0) == WORKSPACE
        assert lib.gdn_workspace_bytes_ssm(ctypes.byref(pr)) > 0
        assert lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(pr)) > 0


@pytest.mark.parametrize("T,H,P,N,G", [(16384, 64, 128, 128, 8), (16384, 80, 64, 128, 1), (131072, 64, 128, 128, 8), (5000, 3, 64, 64, 3)])
def test_scan_workspace_has_no_state_for_a_short_sequence(lib, T, H, P, N, G):
    # only sequences of several segments leave end states: at most twice as many
    # places as one long sequence has, whatever the number of sequences
    one = lib.gdn_workspace_bytes_ssm(ctypes.byref(packed_scan(T, 1, H, P, N, G)))
    assert one > 0
    for n in (2, 9, 256, 2048):
        assert one <= lib.gdn_workspace_bytes_ssm(ctypes.byref(packed_scan(T, n, H, P, N, G))) <= 2 * one, n
    # and none where no sequence can have two
    assert lib.gdn_workspace_bytes_ssm(ctypes.byref(packed_scan(200, 7, H, P, N, G))) == 0


@pytest.mark.parametrize("T,H,P,N,G", [(16384, 64, 128, 128, 8), (16384, 80, 64, 128, 1), (131072, 64, 128, 128, 8), (5000, 3, 64, 64, 3)])
def test_scan_backward_workspace_has_no_state_for_a_short_sequence(lib, T, H, P, N, G):
    # a sequence brings at most one more chunk of the heads' shares of dB and dC (64 x N
    # fp32 a block of columns), its sums, and end states as above
    size = lambda n: lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(packed_scan(T, n, H, P, N, G)))  # noqa: E731
    blocks = H if P == 128 or (H // G) % 2 else H // 2
    ends = 2 * lib.gdn_workspace_bytes_ssm(ctypes.byref(packed_scan(T, 1, H, P, N, G)))
    for n in (2, 9, 256, 2048):
        assert size(n) - size(1) <= (n - 1) * (blocks * 64 * N * 4 + 64 * H) + ends, n


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def test_binding_wants_device_tensors():
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: gdn.norm_forward(x, w), lambda: gdn.norm_backward(x, x, w),
                 lambda: gdn.conv_forward(x[None], torch.zeros(8, 4)), lambda: gdn.conv_step(x, x, torch.zeros(8, 4)),
                 lambda: gdn.ssm_forward(x[None, None], x, w, x, x)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError, match="Tensor"):
        gdn.norm_forward([1.0], w)
