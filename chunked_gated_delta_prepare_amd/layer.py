"""Binding of libgdn's layer operators (include/libgdn_layer.h): the
root-mean-square norm, the short causal convolution and the selective state
space scan around the recurrence.  As in the package itself every step runs in
libgdn's HIP kernels; this module checks tensors, allocates outputs and
workspaces with torch and passes raw pointers and a stream.

    norm_forward(x, weight, residual=None)        -> (y, s, scales)
    norm_backward(dy, s, weight, dres=None)       -> (ds, dx, dweight)
    conv_forward(x, weight, bias=None)            -> (y, final_state)
    conv_backward(dy, x, weight, bias=None)       -> (dx, dweight, dbias, dinitial)
    conv_step(x, state, weight, bias=None)        -> y, the state in place
    ssm_forward(x, dt, A, B, C, D, dt_bias, h0)   -> (y, hT)
    ssm_backward(dy, x, dt, A, B, C, D, dt_bias, h0)
                        -> (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0)
    ssm_step(x, dt, A, B, C, state, D, dt_bias)   -> y, the state in place

The work goes to ``stream``, or to the current stream of the tensors' device;
outputs and workspaces are allocated on that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

GDN_E4M3 = 2
LAYER_EXPORTS = ["gdn_norm_forward", "gdn_norm_backward", "gdn_workspace_bytes_norm_backward",
                 "gdn_conv_forward", "gdn_conv_backward", "gdn_workspace_bytes_conv_backward",
                 "gdn_conv_step", "gdn_ssm_forward", "gdn_workspace_bytes_ssm", "gdn_ssm_backward",
                 "gdn_workspace_bytes_ssm_backward", "gdn_ssm_step"]

_I64, _I32, _F32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", _I64), ("D", _I64), ("x_stride", _I64), ("x_dtype", _I32), ("s_dtype", _I32),
                ("w_dtype", _I32), ("out_dtype", _I32), ("group", _I32), ("eps", _F32)]


class ConvProblem(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("D", _I64), ("W", _I64), ("x_stride_b", _I64),
                ("x_stride_t", _I64), ("dy_stride_b", _I64), ("dy_stride_t", _I64), ("n_seqs", _I64),
                ("io_dtype", _I32), ("w_dtype", _I32), ("silu", _I32)]


class SsmProblem(ctypes.Structure):
    _fields_ = [("B", _I64), ("T", _I64), ("H", _I64), ("P", _I64), ("N", _I64), ("G", _I64),
                ("x_stride_b", _I64), ("x_stride_t", _I64), ("bc_stride_b", _I64), ("bc_stride_t", _I64),
                ("dt_stride_b", _I64), ("dt_stride_t", _I64), ("dxbc_stride_b", _I64),
                ("dxbc_stride_t", _I64), ("n_seqs", _I64), ("io_dtype", _I32), ("dt_dtype", _I32),
                ("softplus", _I32)]


_FP8 = torch.float8_e4m3fn
_CODE = {torch.float32: 0, torch.bfloat16: 1, _FP8: GDN_E4M3}


def declare(lib):
    """Argument types of the layer operators' functions."""
    vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
    n, c, s = (ctypes.POINTER(t) for t in (NormProblem, ConvProblem, SsmProblem))
    lib.gdn_norm_forward.argtypes = [n] + [vp] * 7
    lib.gdn_norm_backward.argtypes = [n] + [vp] * 8 + [sz, vp]
    lib.gdn_conv_forward.argtypes = [c] + [vp] * 8
    lib.gdn_conv_backward.argtypes = [c] + [vp] * 12 + [sz, vp]
    lib.gdn_conv_step.argtypes = [c] + [vp] * 5 + [i64, vp, vp]
    lib.gdn_ssm_forward.argtypes = [s] + [vp] * 12 + [sz, vp]
    lib.gdn_ssm_backward.argtypes = [s] + [vp] * 20 + [sz, vp]
    lib.gdn_ssm_step.argtypes = [s] + [vp] * 9 + [i64, vp, vp]
    for name, arg in (("norm_backward", n), ("conv_backward", c), ("ssm", s), ("ssm_backward", s)):
        f = getattr(lib, "gdn_workspace_bytes_" + name)
        f.argtypes, f.restype = [arg], sz
    for name in LAYER_EXPORTS:
        if "workspace" not in name:
            getattr(lib, name).restype = ctypes.c_int


def _library():
    from . import load_library
    return load_library()


def _call(name, *args):
    lib = _library()
    rc = getattr(lib, name)(*args)
    if rc != 0:
        from . import GdnError
        raise GdnError(name, rc, lib.gdn_status_str(rc).decode())


def _io_code(t, name):
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return _CODE[t.dtype]


def _check(t, name, device, shape, dtype=None, dense=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device or not t.is_cuda:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if dense and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device (HIP) tensor" % name)
    return t.device


class _On:
    """Makes the tensors' device and the stream that the work goes to current,
    so that what is allocated inside belongs to that stream; ``handle`` is the
    stream's."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
        index = device.index
        if stream is None:
            self.handle = torch.cuda.current_stream(index).cuda_stream
            self.ctx = contextlib.nullcontext() if torch.cuda.current_device() == index else torch.cuda.device(index)
        else:
            self.handle = stream.cuda_stream
            self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        return self.ctx.__exit__(*exc)


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _apart(out, name, *inputs):
    """Outputs do not alias inputs."""
    if out is not None and out.numel():
        lo = out.data_ptr()
        hi = lo + out.element_size() * (1 + sum((n - 1) * s for n, s in zip(out.shape, out.stride())))
        for t in inputs:
            if t is not None and t.numel():
                a = t.data_ptr()
                b = a + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
                if a < hi and lo < b:
                    raise ValueError("%s must not share memory with an input" % name)


def _workspace(need, device, workspace):
    if workspace is None:
        workspace = torch.empty(need, device=device, dtype=torch.uint8) if need else None
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())


def _out(t, name, device, shape, dtype, inputs):
    if t is None:
        return torch.empty(shape, device=device, dtype=dtype)
    _check(t, name, device, shape, dtype)
    _apart(t, name, *inputs)
    return t


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def _rows(t):
    """A tensor as rows of its last dimension at one stride: (rows, stride), or
    None if its leading dimensions do not merge."""
    D = t.shape[-1]
    rows = t.numel() // D if D else 0
    if t.dim() == 1:
        return 1, D
    if D > 1 and t.stride(-1) != 1 and rows:
        return None
    stride, want = None, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != want:
            return None
        want = s * n
    return rows, D if stride is None else stride


def norm_forward(x, weight, residual=None, *, eps=1e-6, out_dtype=None, group=0, y=None, s=None,
                 scales=None, stream=None):
    """s = x + residual (in the residual's type), y = s r weight with
    r = 1 / sqrt(mean(s^2) + eps) over the last dimension.

    x [..., D] bf16 or fp32 (rows may be strided); weight [D] in x's type or
    fp32; residual like x, in x's type or fp32.  out_dtype: x's type, or
    torch.float8_e4m3fn with one scale per row (group 0) or per 128 columns
    (group 128): y holds values / scale.  Returns (y, s, scales): s is
    None without a residual, scales [..., groups] fp32 or None.  A given s
    may be the residual."""
    dev = _device(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1, got %s" % (tuple(x.shape),))
    D = x.shape[-1]
    code = _io_code(x, "x")
    merged = _rows(x)
    if merged is None:
        raise ValueError("x's rows must be contiguous and lie at one stride")
    _check(weight, "weight", dev, (D,), (x.dtype, torch.float32))
    sdt = x.dtype
    if residual is not None:
        _check(residual, "residual", dev, x.shape, (x.dtype, torch.float32))
        sdt = residual.dtype
    od = out_dtype or x.dtype
    if od not in (x.dtype, _FP8):
        raise TypeError("out_dtype must be %s or %s, got %s" % (x.dtype, _FP8, od))
    if group not in (0, 128):
        raise ValueError("group must be 0 (a scale per row) or 128, got %r" % (group,))
    with _On(dev, stream) as handle:
        y = _out(y, "y", dev, x.shape, od, (x, weight, residual))
        if residual is not None and (s is None or s.data_ptr() != residual.data_ptr()):
            s = _out(s, "s", dev, x.shape, sdt, (x, weight, residual, y))
        elif residual is not None:
            _check(s, "s", dev, x.shape, sdt)
        if od == _FP8:
            ng = (D + group - 1) // group if group else 1
            scales = _out(scales, "scales", dev, tuple(x.shape[:-1]) + (ng,), torch.float32, (x, weight, residual, y))
        else:
            scales = None
        pr = NormProblem(merged[0], D, merged[1], code, _CODE[sdt], _CODE[weight.dtype], _CODE[od], group, eps)
        _call("gdn_norm_forward", ctypes.byref(pr), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y),
              _ptr(s) if residual is not None else None, _ptr(scales), handle)
    return y, (None if residual is None else s), scales


def norm_backward(dy, s, weight, dres=None, *, eps=1e-6, x_dtype=None, ds=None, dx=None, dweight=None,
                  workspace=None, stream=None):
    """The norm's gradients from dy [..., D] (of y, in x's type), s as
    norm_forward returned it (x where there was no residual), and dres (of s, in s's type, or None).  Returns
    (ds, dx, dweight): ds in s's type is the gradient of the residual; dx in
    x_dtype (default: dy's type) is that of x, ds itself where the types are
    equal; dweight [D] fp32.  A given ds may be dres."""
    dev = _device(dy, "dy")
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError("dy must have a last dimension of at least 1, got %s" % (tuple(dy.shape),))
    D = dy.shape[-1]
    code = _io_code(dy, "dy")
    if x_dtype not in (None, dy.dtype):
        raise TypeError("dy has x's type: got %s for x of %s" % (dy.dtype, x_dtype))
    _check(dy, "dy", dev, dy.shape)
    _check(s, "s", dev, dy.shape, (dy.dtype, torch.float32))
    _check(weight, "weight", dev, (D,), (dy.dtype, torch.float32))
    if dres is not None:
        _check(dres, "dres", dev, dy.shape, s.dtype)
    lib = _library()
    with _On(dev, stream) as handle:
        ins = (dy, s, weight)
        if dres is not None and ds is not None and ds.data_ptr() == dres.data_ptr():
            _check(ds, "ds", dev, dy.shape, s.dtype)
        else:
            ds = _out(ds, "ds", dev, dy.shape, s.dtype, ins + (dres,))
        if s.dtype == dy.dtype:
            if dx is not None and dx is not ds:
                raise ValueError("dx is ds where x and s have one type")
            dx = ds
        else:
            dx = _out(dx, "dx", dev, dy.shape, dy.dtype, ins + (dres, ds))
        dweight = _out(dweight, "dweight", dev, (D,), torch.float32, ins + (dres, ds, dx))
        pr = NormProblem(dy.numel() // D, D, D, code, _CODE[s.dtype], _CODE[weight.dtype], code, 0, eps)
        need = int(lib.gdn_workspace_bytes_norm_backward(ctypes.byref(pr)))
        workspace, size = _workspace(need, dev, workspace)
        _call("gdn_norm_backward", ctypes.byref(pr), _ptr(dy), _ptr(s), _ptr(weight), _ptr(dres), _ptr(ds),
              None if dx is ds else _ptr(dx), _ptr(dweight), _ptr(workspace), size, handle)
    return ds, dx, dweight


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def _silu(activation):
    if activation not in ("silu", None):
        raise ValueError("activation must be 'silu' or None, got %r" % (activation,))
    return 1 if activation == "silu" else 0


def _strides(t, name):
    """(batch, token) strides of [B, T, ...] whose other dimensions are dense."""
    want = 1
    for n, s in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        if n != 1 and s != want and t.numel():
            raise ValueError("%s must be contiguous behind its token dimension" % name)
        want *= n
    return (t.stride(0) if t.shape[0] != 1 else 0), (t.stride(1) if t.shape[1] != 1 else want)


def _packed(cu, dev, B):
    if cu is None:
        return 0
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.numel() < 2:
        raise ValueError("cu_seqlens must hold N + 1 >= 2 offsets")
    _check(cu, "cu_seqlens", dev, (cu.numel(),), torch.int32)
    if B != 1:
        raise ValueError("packed sequences use a batch of 1, got %d" % B)
    return cu.numel() - 1


def _conv_checks(x, weight, bias):
    dev = _device(x, "x")
    code = _io_code(x, "x")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    D, W = x.shape[-1], weight.shape[1]
    if W not in (2, 3, 4):
        raise ValueError("weight must have 2, 3 or 4 taps, got %d" % W)
    _check(weight, "weight", dev, (D, W), (x.dtype, torch.float32))
    if bias is not None:
        _check(bias, "bias", dev, (D,), weight.dtype)
    return dev, code, D, W


def conv_forward(x, weight, bias=None, *, activation="silu", initial_state=None, cu_seqlens=None, y=None,
                 final_state=None, output_final_state=True, stream=None):
    """y_t = act(bias + sum_j weight[:, j] x_{t - (W-1) + j}) per channel, over
    the tokens of each sequence: x [B, T, D] (tokens may be strided), weight
    [D, W] with W 2 to 4, bias [D]; both in x's type or fp32.  States hold the
    last W - 1 inputs: [B, W-1, D], or [N, W-1, D] with cu_seqlens (int32, N + 1
    offsets, a batch of 1).  Returns (y, final_state or None)."""
    dev, code, D, W = _conv_checks(x, weight, bias)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D], got %s" % (tuple(x.shape),))
    B, T, _ = x.shape
    n = _packed(cu_seqlens, dev, B)
    st = (n or B, W - 1, D)
    if initial_state is not None:
        _check(initial_state, "initial_state", dev, st, x.dtype)
    sb, stt = _strides(x, "x")
    silu = _silu(activation)
    with _On(dev, stream) as handle:
        ins = (x, weight, bias, initial_state, cu_seqlens)
        y = _out(y, "y", dev, (B, T, D), x.dtype, ins)
        if final_state is not None or output_final_state:
            final_state = _out(final_state, "final_state", dev, st, x.dtype, ins + (y,))
        pr = ConvProblem(B, T, D, W, sb, stt, 0, 0, n, code, _CODE[weight.dtype], silu)
        _call("gdn_conv_forward", ctypes.byref(pr), _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state),
              _ptr(cu_seqlens), _ptr(y), _ptr(final_state), handle)
    return y, final_state


def conv_backward(dy, x, weight, bias=None, *, activation="silu", initial_state=None, cu_seqlens=None,
                  dfinal=None, dx=None, dweight=None, dbias=None, dinitial=None, workspace=None, stream=None):
    """The convolution's gradients for dy [B, T, D] (tokens may be strided) and
    dfinal (of the final states, or None).  Returns (dx, dweight [D, W] fp32,
    dbias [D] fp32 or None, dinitial or None): dbias with a bias, dinitial
    with an initial_state."""
    dev, code, D, W = _conv_checks(x, weight, bias)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D], got %s" % (tuple(x.shape),))
    B, T, _ = x.shape
    _check(dy, "dy", dev, (B, T, D), x.dtype, dense=False)
    n = _packed(cu_seqlens, dev, B)
    st = (n or B, W - 1, D)
    for t, name in ((initial_state, "initial_state"), (dfinal, "dfinal")):
        if t is not None:
            _check(t, name, dev, st, x.dtype)
    sb, stt = _strides(x, "x")
    gb, gt = _strides(dy, "dy")
    silu = _silu(activation)
    lib = _library()
    with _On(dev, stream) as handle:
        ins = (dy, x, weight, bias, initial_state, cu_seqlens, dfinal)
        dx = _out(dx, "dx", dev, (B, T, D), x.dtype, ins)
        dweight = _out(dweight, "dweight", dev, (D, W), torch.float32, ins + (dx,))
        if bias is not None:
            dbias = _out(dbias, "dbias", dev, (D,), torch.float32, ins + (dx, dweight))
        if initial_state is not None:
            dinitial = _out(dinitial, "dinitial", dev, st, x.dtype, ins + (dx, dweight, dbias))
        pr = ConvProblem(B, T, D, W, sb, stt, gb, gt, n, code, _CODE[weight.dtype], silu)
        workspace, size = _workspace(int(lib.gdn_workspace_bytes_conv_backward(ctypes.byref(pr))), dev, workspace)
        _call("gdn_conv_backward", ctypes.byref(pr), _ptr(dy), _ptr(x), _ptr(weight), _ptr(bias),
              _ptr(initial_state), _ptr(cu_seqlens), _ptr(dfinal), _ptr(dx), _ptr(dweight),
              _ptr(dbias) if bias is not None else None, _ptr(dinitial) if initial_state is not None else None,
              _ptr(workspace), size, handle)
    return dx, dweight, dbias if bias is not None else None, dinitial if initial_state is not None else None


def _slots(slots, dev, B):
    if slots is not None:
        _check(slots, "slots", dev, (B,), torch.int32)


def conv_step(x, state, weight, bias=None, *, activation="silu", slots=None, y=None, stream=None):
    """One token for each of B sequences: x [B, D] (rows may be strided),
    state [S, W-1, D] in x's type, moved on in place; slots [B] int32 names
    each row's state (None: row b has state b).  A row whose slot is outside
    [0, S), or that an earlier row names already, is padding: its y is zero
    and no state changes.  Returns y [B, D]."""
    dev, code, D, W = _conv_checks(x, weight, bias)
    if x.dim() != 2:
        raise ValueError("x must be [B, D], got %s" % (tuple(x.shape),))
    B = x.shape[0]
    if B and D > 1 and x.stride(1) != 1:
        raise ValueError("x's rows must be contiguous")
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [S, W-1, D]")
    _check(state, "state", dev, (state.shape[0], W - 1, D), x.dtype)
    _slots(slots, dev, B)
    _apart(state, "state", x, weight, bias, slots)
    silu = _silu(activation)
    with _On(dev, stream) as handle:
        y = _out(y, "y", dev, (B, D), x.dtype, (x, weight, bias, state, slots))
        if B:
            pr = ConvProblem(B, 1, D, W, x.stride(0) if B > 1 else D, D, 0, 0, 0, code, _CODE[weight.dtype], silu)
            _call("gdn_conv_step", ctypes.byref(pr), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(slots),
                  state.shape[0], _ptr(y), handle)
    return y


# ---------------------------------------------------------------------------
# selective state space scan
# ---------------------------------------------------------------------------

def _ssm_checks(x, dt, A, B, C, D, dt_bias, lead):
    """Types and shapes of a scan's inputs; lead dimensions before [H, P]."""
    dev = _device(x, "x")
    code = _io_code(x, "x")
    if x.dim() != lead + 2 or not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError("x and B must have %d dimensions" % (lead + 2))
    H, P = x.shape[-2:]
    G, N = B.shape[-2:]
    _check(B, "B", dev, tuple(x.shape[:lead]) + (G, N), x.dtype, dense=False)
    _check(C, "C", dev, B.shape, x.dtype, dense=False)
    _check(dt, "dt", dev, tuple(x.shape[:lead]) + (H,), (x.dtype, torch.float32), dense=False)
    _check(A, "A", dev, (H,), torch.float32)
    for t, name in ((D, "D"), (dt_bias, "dt_bias")):
        if t is not None:
            _check(t, name, dev, (H,), torch.float32)
    return dev, code, H, P, G, N


def _ssm_problem(x, dt, B, C, code, softplus, n, grads=(0, 0)):
    H, P = x.shape[-2:]
    G, N = B.shape[-2:]
    sb, sc = _strides(B, "B"), _strides(C, "C")
    if sb != sc:
        raise ValueError("B and C must have the same strides, got %s and %s" % (sb, sc))
    return SsmProblem(x.shape[0], x.shape[1], H, P, N, G, *_strides(x, "x"), *sb, *_strides(dt, "dt"), *grads, n,
                      code, _CODE[dt.dtype], 1 if softplus else 0)


def ssm_forward(x, dt, A, B, C, D=None, dt_bias=None, h0=None, *, dt_softplus=True, cu_seqlens=None, y=None,
                hT=None, output_final_state=True, workspace=None, stream=None):
    """Selective state space scan: h_t = e^(dt_t A) h_{t-1} + dt_t B_t x_t^T,
    y_t = h_t^T C_t + D x_t, dt = softplus(dt + dt_bias) (or without softplus).

    x [b, T, H, P], B and C [b, T, G, N] (tokens may be strided, rows 16-byte
    aligned), P and N 64 or 128, H a multiple of G; dt [b, T, H] in x's type or
    fp32; A, D, dt_bias [H] fp32; h0 [b, H, N, P] fp32, or [n, H, N, P] with
    cu_seqlens (as in conv_forward).  Returns (y [b, T, H, P], hT like h0 or
    None)."""
    dev, code, H, P, G, N = _ssm_checks(x, dt, A, B, C, D, dt_bias, 2)
    n = _packed(cu_seqlens, dev, x.shape[0])
    st = (n or x.shape[0], H, N, P)
    if h0 is not None:
        _check(h0, "h0", dev, st, torch.float32)
    pr = _ssm_problem(x, dt, B, C, code, dt_softplus, n)
    lib = _library()
    with _On(dev, stream) as handle:
        ins = (x, dt, A, B, C, D, dt_bias, h0, cu_seqlens)
        y = _out(y, "y", dev, x.shape, x.dtype, ins)
        if hT is not None or output_final_state:
            hT = _out(hT, "hT", dev, st, torch.float32, ins + (y,))
        workspace, size = _workspace(int(lib.gdn_workspace_bytes_ssm(ctypes.byref(pr))), dev, workspace)
        _call("gdn_ssm_forward", ctypes.byref(pr), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
              _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), _ptr(y), _ptr(hT), _ptr(workspace), size, handle)
    return y, hT


def ssm_backward(dy, x, dt, A, B, C, D=None, dt_bias=None, h0=None, dhT=None, *, dt_softplus=True,
                 cu_seqlens=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dD=None, ddt_bias=None, dh0=None,
                 workspace=None, stream=None):
    """The scan's gradients for dy [b, T, H, P] and dhT (of the final states,
    or None); the states are formed again from the inputs.  Returns (dx, ddt,
    dA, dB, dC, dD, ddt_bias, dh0): dx, dB and dC in x's type, ddt in dt's, the
    others fp32; dD, ddt_bias and dh0 are None where D, dt_bias and h0 are.
    dx, dB and dC may be given as parts of one buffer (with the same strides
    between tokens), as the gradient of a convolution's output."""
    dev, code, H, P, G, N = _ssm_checks(x, dt, A, B, C, D, dt_bias, 2)
    b, T = x.shape[:2]
    n = _packed(cu_seqlens, dev, b)
    st = (n or b, H, N, P)
    _check(dy, "dy", dev, x.shape, x.dtype)
    for t, name in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _check(t, name, dev, st, torch.float32)
    lib = _library()
    ins = (dy, x, dt, A, B, C, D, dt_bias, h0, dhT, cu_seqlens)
    with _On(dev, stream) as handle:
        given = [t is not None for t in (dx, dB, dC)]
        if any(given):
            if not all(given):
                raise ValueError("dx, dB and dC are given together or not at all")
            for t, name, like in ((dx, "dx", x), (dB, "dB", B), (dC, "dC", C)):
                _check(t, name, dev, like.shape, x.dtype, dense=False)
            grads = _strides(dx, "dx")
            if any(_strides(t, name) != grads for t, name in ((dB, "dB"), (dC, "dC"))):
                raise ValueError("dx, dB and dC must have the same strides between batches and tokens")
            lo = min(t.data_ptr() for t in (dx, dB, dC))
            for t in ins:
                if t is not None and t.numel() and T and lo < t.data_ptr() + t.numel() * t.element_size():
                    for o, name in ((dx, "dx"), (dB, "dB"), (dC, "dC")):
                        _apart(o, name, t)
        else:
            # side by side, as the convolution that feeds the scan laid them out
            both = torch.empty(b, T, H * P + 2 * G * N, device=dev, dtype=x.dtype)
            dx = both[..., :H * P].unflatten(-1, (H, P))
            dB = both[..., H * P:H * P + G * N].unflatten(-1, (G, N))
            dC = both[..., H * P + G * N:].unflatten(-1, (G, N))
            grads = _strides(dx, "dx")
        ddt = _out(ddt, "ddt", dev, (b, T, H), dt.dtype, ins)
        dA = _out(dA, "dA", dev, (H,), torch.float32, ins)
        if D is not None:
            dD = _out(dD, "dD", dev, (H,), torch.float32, ins)
        if dt_bias is not None:
            ddt_bias = _out(ddt_bias, "ddt_bias", dev, (H,), torch.float32, ins)
        if h0 is not None:
            dh0 = _out(dh0, "dh0", dev, st, torch.float32, ins)
        pr = _ssm_problem(x, dt, B, C, code, dt_softplus, n, grads)
        workspace, size = _workspace(int(lib.gdn_workspace_bytes_ssm_backward(ctypes.byref(pr))), dev, workspace)
        _call("gdn_ssm_backward", ctypes.byref(pr), _ptr(dy), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
              _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), _ptr(dhT), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC),
              _ptr(dD) if D is not None else None, _ptr(ddt_bias) if dt_bias is not None else None,
              _ptr(dh0) if h0 is not None else None, _ptr(workspace), size, handle)
    return (dx, ddt, dA, dB, dC, dD if D is not None else None, ddt_bias if dt_bias is not None else None,
            dh0 if h0 is not None else None)


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, dt_softplus=True, slots=None, y=None, stream=None):
    """One token for each of b sequences: x [b, H, P], dt [b, H], B and C
    [b, G, N] (rows may be strided); state [S, H, N, P] fp32, moved on in place;
    slots as in conv_step.  Returns y [b, H, P]."""
    dev, code, H, P, G, N = _ssm_checks(x, dt, A, B, C, D, dt_bias, 1)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [S, H, N, P]")
    _check(state, "state", dev, (state.shape[0], H, N, P), torch.float32)
    b = x.shape[0]
    _slots(slots, dev, b)
    ins = (x, dt, A, B, C, D, dt_bias, slots)
    _apart(state, "state", *ins)
    with _On(dev, stream) as handle:
        y = _out(y, "y", dev, x.shape, x.dtype, ins + (state,))
        if b:
            # a row is a batch of one token
            pr = _ssm_problem(x[:, None], dt[:, None], B[:, None], C[:, None], code, dt_softplus, 0)
            _call("gdn_ssm_step", ctypes.byref(pr), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                  _ptr(dt_bias), _ptr(state), _ptr(slots), state.shape[0], _ptr(y), handle)
    return y
