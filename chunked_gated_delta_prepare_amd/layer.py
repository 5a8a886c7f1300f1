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

import ctypes
import functools

import torch

from .layer_abi import (GDN_E4M3, LAYER_EXPORTS, ConvProblem, NormProblem,  # noqa: F401
                        SsmProblem, declare)

_FP8 = torch.float8_e4m3fn
_CODE = {torch.float32: 0, torch.bfloat16: 1, _FP8: GDN_E4M3}

_functions = {}


def _function(name):
    f = _functions.get(name)
    if f is None:
        from . import load_library
        f = _functions[name] = getattr(load_library(), name)
    return f


def _call(name, *args):
    rc = (_functions.get(name) or _function(name))(*args)
    if rc != 0:
        from . import GdnError, load_library
        raise GdnError(name, rc, load_library().gdn_status_str(rc).decode())


# What a problem's sizes, strides and types alone decide: its structure and
# the bytes of workspace it needs.
@functools.lru_cache(maxsize=4096)
def _problem(kind, size_of, *fields):
    ref = ctypes.byref(kind(*fields))
    return ref, int(_function(size_of)(ref)) if size_of else 0


def _io_code(t, name):
    code = _CODE.get(t.dtype)
    if code is None or code == GDN_E4M3:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return code


def _check(t, name, device, shape, dtype=None, other=None, dense=True):
    """A tensor on the device, of this shape, and of dtype or other."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if dtype is not None and t.dtype is not dtype and t.dtype is not other:
        raise TypeError("%s must be %s, got %s" % (name, dtype if other in (None, dtype) else "%s or %s" % (dtype, other), t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if dense and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device (HIP) tensor" % name)
    return t.device


def _on(device, stream, work, *args):
    """work(handle, *args) with the tensors' device current, and the stream that
    the work goes to, so that what is allocated in it belongs to that stream;
    handle is the stream's."""
    index = device.index
    if stream is None:
        if torch._C._cuda_getDevice() == index:
            return work(torch._C._cuda_getCurrentRawStream(index), *args)
        with torch.cuda.device(index):
            return work(torch._C._cuda_getCurrentRawStream(index), *args)
    if stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        return work(stream.cuda_stream, *args)


def _ptr(t):
    return None if t is None else t.data_ptr() or None


def _span(t):
    """The addresses a tensor reaches, [first, last + 1)."""
    lo = t.data_ptr()
    if t.is_contiguous():
        return lo, lo + t.nbytes
    return lo, lo + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _apart(out, name, *inputs):
    """Outputs do not alias inputs."""
    if out is not None and out.nbytes:
        lo, hi = _span(out)
        for t in inputs:
            if t is None:
                continue
            # (as few calls to torch as it takes: the steps have eight inputs)
            a = t.data_ptr()
            if a < hi and not (a + t.nbytes <= lo and t.is_contiguous()) and lo < _span(t)[1] and t.nbytes:
                raise ValueError("%s must not share memory with an input" % name)


def _workspace(need, device, workspace):
    if workspace is None:
        workspace = torch.empty(need, device=device, dtype=torch.uint8) if need else None
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())


def _unwritten(t, name, without):
    """A given output that the call has no values for."""
    if t is not None:
        raise ValueError("%s is not written without %s" % (name, without))


def _out(t, name, device, shape, dtype, inputs, like=None):
    """A given output, checked, or a new one; like: a tensor of its shape, if there
    is one (a call less to torch's slower ways)."""
    if t is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like, dtype=dtype)
        return torch.empty(tuple(shape), device=device, dtype=dtype)
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
    if D > 1 and t.stride(-1) != 1 and rows:
        return None
    if t.dim() == 1:
        return 1, D
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
    shape, dt = x.shape, x.dtype
    if x.dim() < 1 or shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1, got %s" % (tuple(shape),))
    code = _io_code(x, "x")
    _check(weight, "weight", dev, shape[-1:], dt, torch.float32)
    if residual is not None:
        _check(residual, "residual", dev, shape, dt, torch.float32)
    if out_dtype not in (None, dt, _FP8):
        raise TypeError("out_dtype must be %s or %s, got %s" % (dt, _FP8, out_dtype))
    if group not in (0, 128):
        raise ValueError("group must be 0 (a scale per row) or 128, got %r" % (group,))
    return _on(dev, stream, _norm_forward, dev, code, x, weight, residual, eps, out_dtype or dt, group, y, s, scales)


def _norm_forward(handle, dev, code, x, weight, residual, eps, od, group, y, s, scales):
    shape, D = x.shape, x.shape[-1]
    if x.is_contiguous():
        rows, stride = x.numel() // D, D
    else:
        merged = _rows(x)
        if merged is None:
            raise ValueError("x's rows must be contiguous and lie at one stride")
        rows, stride = merged
    y = _out(y, "y", dev, shape, od, (x, weight, residual), x)
    scode = code
    if residual is not None:
        scode = _CODE[residual.dtype]
        if s is not None and s.data_ptr() == residual.data_ptr():
            _check(s, "s", dev, shape, residual.dtype)
            _apart(s, "s", x, weight, y)
        else:
            s = _out(s, "s", dev, shape, residual.dtype, (x, weight, residual, y), residual)
    else:
        _unwritten(s, "s", "a residual")
    if od is _FP8:
        scales = _out(scales, "scales", dev, shape[:-1] + ((D + group - 1) // group if group else 1,), torch.float32,
                      (x, weight, residual, y, s))
    else:
        _unwritten(scales, "scales", "an 8-bit output")
    pr, _ = _problem(NormProblem, None, rows, D, stride, code, scode, _CODE[weight.dtype], _CODE[od], group, eps)
    _call("gdn_norm_forward", pr, x.data_ptr(), _ptr(residual), weight.data_ptr(), y.data_ptr(), _ptr(s), _ptr(scales), handle)
    return y, s, scales


def norm_backward(dy, s, weight, dres=None, *, eps=1e-6, x_dtype=None, ds=None, dx=None, dweight=None,
                  workspace=None, stream=None):
    """The norm's gradients from dy [..., D] (of y, in x's type), s as
    norm_forward returned it (x where there was no residual), and dres (of s, in
    s's type, or None).  Returns (ds, dx, dweight): ds in s's type is the
    gradient of the residual; dx in x_dtype (default: dy's type) is that of x,
    ds itself where the types are equal; dweight [D] fp32.  A given ds may be
    dres."""
    dev = _device(dy, "dy")
    shape, dt = dy.shape, dy.dtype
    if dy.dim() < 1 or shape[-1] < 1:
        raise ValueError("dy must have a last dimension of at least 1, got %s" % (tuple(shape),))
    code = _io_code(dy, "dy")
    if x_dtype not in (None, dt):
        raise TypeError("dy has x's type: got %s for x of %s" % (dt, x_dtype))
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    _check(s, "s", dev, shape, dt, torch.float32)
    _check(weight, "weight", dev, shape[-1:], dt, torch.float32)
    if dres is not None:
        _check(dres, "dres", dev, shape, s.dtype)
    return _on(dev, stream, _norm_backward, dev, code, dy, s, weight, dres, eps, ds, dx, dweight, workspace)


def _norm_backward(handle, dev, code, dy, s, weight, dres, eps, ds, dx, dweight, workspace):
    shape, D = dy.shape, dy.shape[-1]
    ins = (dy, s, weight)
    if dres is not None and ds is not None and ds.data_ptr() == dres.data_ptr():
        _check(ds, "ds", dev, shape, s.dtype)
        _apart(ds, "ds", *ins)
    else:
        ds = _out(ds, "ds", dev, shape, s.dtype, ins + (dres,), s)
    if s.dtype is dy.dtype:
        if dx is not None and dx is not ds:
            raise ValueError("dx is ds where x and s have one type")
        dx = None
    else:
        dx = _out(dx, "dx", dev, shape, dy.dtype, ins + (dres, ds), dy)
    dweight = _out(dweight, "dweight", dev, shape[-1:], torch.float32, ins + (dres, ds, dx))
    pr, need = _problem(NormProblem, "gdn_workspace_bytes_norm_backward", dy.numel() // D, D, D, code, _CODE[s.dtype],
                        _CODE[weight.dtype], code, 0, eps)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_norm_backward", pr, dy.data_ptr(), s.data_ptr(), weight.data_ptr(), _ptr(dres), ds.data_ptr(), _ptr(dx), dweight.data_ptr(),
          _ptr(workspace), size, handle)
    return ds, ds if dx is None else dx, dweight


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def _silu(activation):
    if activation not in ("silu", None):
        raise ValueError("activation must be 'silu' or None, got %r" % (activation,))
    return 1 if activation == "silu" else 0


def _strides(t, name):
    """(batch, token) strides of [B, T, D] or [B, T, H, D] whose tokens are dense."""
    shape, strides = t.shape, t.stride()
    row = shape[-1]
    dense = row == 1 or strides[-1] == 1
    if len(shape) == 4:
        dense = dense and (shape[2] == 1 or strides[2] == row)
        row *= shape[2]
    if not dense and t.numel():
        raise ValueError("%s must be contiguous behind its token dimension" % name)
    return (strides[0] if shape[0] != 1 else 0), (strides[1] if shape[1] != 1 else row)


def _packed(cu, dev, B):
    if cu is None:
        return 0
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu_seqlens must hold N + 1 >= 2 offsets")
    _check(cu, "cu_seqlens", dev, cu.shape, torch.int32)
    if B != 1:
        raise ValueError("packed sequences use a batch of 1, got %d" % B)
    return cu.shape[0] - 1


def _conv_checks(x, weight, bias, dims):
    dev = _device(x, "x")
    code = _io_code(x, "x")
    if x.dim() != dims:
        raise ValueError("x must be %s, got %s" % ("[B, T, D]" if dims == 3 else "[B, D]", tuple(x.shape)))
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    D, W = x.shape[-1], weight.shape[1]
    if W not in (2, 3, 4):
        raise ValueError("weight must have 2, 3 or 4 taps, got %d" % W)
    _check(weight, "weight", dev, (D, W), x.dtype, torch.float32)
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
    dev, code, D, W = _conv_checks(x, weight, bias, 3)
    n = _packed(cu_seqlens, dev, x.shape[0])
    if initial_state is not None:
        _check(initial_state, "initial_state", dev, (n or x.shape[0], W - 1, D), x.dtype)
    return _on(dev, stream, _conv_forward, dev, code, x, weight, bias, _silu(activation), initial_state, cu_seqlens, n, y,
               final_state, output_final_state)


def _conv_forward(handle, dev, code, x, weight, bias, silu, initial_state, cu_seqlens, n, y, final_state, want):
    B, T, D = x.shape
    W = weight.shape[1]
    ins = (x, weight, bias, initial_state, cu_seqlens)
    y = _out(y, "y", dev, x.shape, x.dtype, ins, x)
    if final_state is not None or want:
        final_state = _out(final_state, "final_state", dev, (n or B, W - 1, D), x.dtype, ins + (y,), initial_state)
    pr, _ = _problem(ConvProblem, None, B, T, D, W, *_strides(x, "x"), 0, 0, n, code, _CODE[weight.dtype], silu)
    _call("gdn_conv_forward", pr, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), y.data_ptr(),
          _ptr(final_state), handle)
    return y, final_state


def conv_backward(dy, x, weight, bias=None, *, activation="silu", initial_state=None, cu_seqlens=None,
                  dfinal=None, dx=None, dweight=None, dbias=None, dinitial=None, workspace=None, stream=None):
    """The convolution's gradients for dy [B, T, D] (tokens may be strided) and
    dfinal (of the final states, or None).  Returns (dx, dweight [D, W] fp32,
    dbias [D] fp32 or None, dinitial or None): dbias with a bias, dinitial
    with an initial_state."""
    dev, code, D, W = _conv_checks(x, weight, bias, 3)
    if bias is None:
        _unwritten(dbias, "dbias", "a bias")
    if initial_state is None:
        _unwritten(dinitial, "dinitial", "an initial_state")
    _check(dy, "dy", dev, x.shape, x.dtype, dense=False)
    n = _packed(cu_seqlens, dev, x.shape[0])
    for t, name in ((initial_state, "initial_state"), (dfinal, "dfinal")):
        if t is not None:
            _check(t, name, dev, (n or x.shape[0], W - 1, D), x.dtype)
    return _on(dev, stream, _conv_backward, dev, code, dy, x, weight, bias, _silu(activation), initial_state, cu_seqlens, n,
               dfinal, dx, dweight, dbias, dinitial, workspace)


def _conv_backward(handle, dev, code, dy, x, weight, bias, silu, initial_state, cu_seqlens, n, dfinal, dx, dweight, dbias,
                   dinitial, workspace):
    B, T, D = x.shape
    W = weight.shape[1]
    ins = (dy, x, weight, bias, initial_state, cu_seqlens, dfinal)
    dx = _out(dx, "dx", dev, x.shape, x.dtype, ins, x)
    dweight = _out(dweight, "dweight", dev, (D, W), torch.float32, ins + (dx,))
    dbias = None if bias is None else _out(dbias, "dbias", dev, (D,), torch.float32, ins + (dx, dweight))
    dinitial = None if initial_state is None else _out(dinitial, "dinitial", dev, initial_state.shape, x.dtype,
                                                       ins + (dx, dweight, dbias))
    pr, need = _problem(ConvProblem, "gdn_workspace_bytes_conv_backward", B, T, D, W, *_strides(x, "x"), *_strides(dy, "dy"),
                        n, code, _CODE[weight.dtype], silu)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_conv_backward", pr, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens),
          _ptr(dfinal), dx.data_ptr(), dweight.data_ptr(), _ptr(dbias), _ptr(dinitial), _ptr(workspace), size, handle)
    return dx, dweight, dbias, dinitial


def conv_step(x, state, weight, bias=None, *, activation="silu", slots=None, y=None, stream=None):
    """One token for each of B sequences: x [B, D] (rows may be strided),
    state [S, W-1, D] in x's type, moved on in place; slots [B] int32 names
    each row's state (None: row b has state b).  A row whose slot is outside
    [0, S), or that an earlier row names already, is padding: its y is zero
    and no state changes.  Returns y [B, D]."""
    dev, code, D, W = _conv_checks(x, weight, bias, 2)
    B = x.shape[0]
    if D > 1 and B and x.stride(1) != 1:
        raise ValueError("x's rows must be contiguous")
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [S, W-1, D]")
    _check(state, "state", dev, (state.shape[0], W - 1, D), x.dtype)
    if slots is not None:
        _check(slots, "slots", dev, (B,), torch.int32)
    _apart(state, "state", x, weight, bias, slots)
    return _on(dev, stream, _conv_step, dev, code, x, state, weight, bias, _silu(activation), slots, y)


def _conv_step(handle, dev, code, x, state, weight, bias, silu, slots, y):
    B, D = x.shape
    y = _out(y, "y", dev, (B, D), x.dtype, (x, weight, bias, state, slots), x)
    if B:
        pr, _ = _problem(ConvProblem, None, B, 1, D, weight.shape[1], x.stride(0) if B > 1 else D, D, 0, 0, 0, code,
                         _CODE[weight.dtype], silu)
        _call("gdn_conv_step", pr, x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(), _ptr(slots), state.shape[0], y.data_ptr(),
              handle)
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
    H = x.shape[-2]
    _check(B, "B", dev, x.shape[:lead] + B.shape[lead:], x.dtype, dense=False)
    _check(C, "C", dev, B.shape, x.dtype, dense=False)
    _check(dt, "dt", dev, x.shape[:-1], x.dtype, torch.float32, dense=False)
    _check(A, "A", dev, (H,), torch.float32)
    if D is not None:
        _check(D, "D", dev, (H,), torch.float32)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", dev, (H,), torch.float32)
    return dev, code


def _bc_strides(B, C):
    sb = _strides(B, "B")
    if _strides(C, "C") != sb:
        raise ValueError("B and C must have the same strides, got %s and %s" % (sb, _strides(C, "C")))
    return sb


def ssm_forward(x, dt, A, B, C, D=None, dt_bias=None, h0=None, *, dt_softplus=True, cu_seqlens=None, y=None,
                hT=None, output_final_state=True, workspace=None, stream=None):
    """Selective state space scan: h_t = e^(dt_t A) h_{t-1} + dt_t B_t x_t^T,
    y_t = h_t^T C_t + D x_t, dt = softplus(dt + dt_bias) (or without softplus).

    x [b, T, H, P], B and C [b, T, G, N] (tokens may be strided, rows 16-byte
    aligned), P and N 64 or 128, H a multiple of G; dt [b, T, H] in x's type or
    fp32; A, D, dt_bias [H] fp32; h0 [b, H, N, P] fp32, or [n, H, N, P] with
    cu_seqlens (as in conv_forward).  A NaN in a token reaches neither the
    tokens before it nor other sequences.  Returns (y [b, T, H, P], hT like h0 or
    None); y does not depend on whether hT is asked for."""
    dev, code = _ssm_checks(x, dt, A, B, C, D, dt_bias, 2)
    n = _packed(cu_seqlens, dev, x.shape[0])
    st = (n or x.shape[0], x.shape[2], B.shape[3], x.shape[3])
    if h0 is not None:
        _check(h0, "h0", dev, st, torch.float32)
    return _on(dev, stream, _ssm_forward, dev, code, x, dt, A, B, C, D, dt_bias, h0, 1 if dt_softplus else 0, cu_seqlens, n,
               st, y, hT, output_final_state, workspace)


def _ssm_forward(handle, dev, code, x, dt, A, B, C, D, dt_bias, h0, softplus, cu_seqlens, n, st, y, hT, want, workspace):
    ins = (x, dt, A, B, C, D, dt_bias, h0, cu_seqlens)
    y = _out(y, "y", dev, x.shape, x.dtype, ins, x)
    if hT is not None or want:
        hT = _out(hT, "hT", dev, st, torch.float32, ins + (y,), h0)
    pr, need = _problem(SsmProblem, "gdn_workspace_bytes_ssm", *x.shape, B.shape[3], B.shape[2], *_strides(x, "x"),
                        *_bc_strides(B, C), *_strides(dt, "dt"), 0, 0, n, code, _CODE[dt.dtype], softplus)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_ssm_forward", pr, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(h0),
          _ptr(cu_seqlens), y.data_ptr(), _ptr(hT), _ptr(workspace), size, handle)
    return y, hT


def ssm_backward(dy, x, dt, A, B, C, D=None, dt_bias=None, h0=None, dhT=None, *, dt_softplus=True,
                 cu_seqlens=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dD=None, ddt_bias=None, dh0=None,
                 workspace=None, stream=None):
    """The scan's gradients for dy [b, T, H, P] and dhT (of the final states,
    or None); the states are formed again from the inputs.  Returns (dx, ddt,
    dA, dB, dC, dD, ddt_bias, dh0): dx, dB and dC in x's type, ddt in dt's, the
    others fp32; dD, ddt_bias and dh0 are None where D, dt_bias and h0 are.
    dx, dB and dC may be given as parts of one buffer (with the same strides
    between batches and between tokens), as the gradient of a convolution's
    output."""
    dev, code = _ssm_checks(x, dt, A, B, C, D, dt_bias, 2)
    n = _packed(cu_seqlens, dev, x.shape[0])
    st = (n or x.shape[0], x.shape[2], B.shape[3], x.shape[3])
    _check(dy, "dy", dev, x.shape, x.dtype)
    for t, name, of, what in ((dD, "dD", D, "D"), (ddt_bias, "ddt_bias", dt_bias, "dt_bias"), (dh0, "dh0", h0, "h0")):
        if of is None:
            _unwritten(t, name, what)
    for t, name in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _check(t, name, dev, st, torch.float32)
    return _on(dev, stream, _ssm_backward, dev, code, dy, x, dt, A, B, C, D, dt_bias, h0, dhT, 1 if dt_softplus else 0,
               cu_seqlens, n, st, (dx, dB, dC), ddt, dA, dD, ddt_bias, dh0, workspace)


def _side_by_side(grads, strides, b, T):
    """dx, dB and dC of one batch and token stride do not overlap."""
    if not grads[0].numel():
        return
    sb, st = strides
    first = sorted((t.data_ptr() // t.element_size(), t[0, 0].numel()) for t in grads)
    end = max(at + n for at, n in first)
    rows = all(a + n <= c for (a, n), (c, _) in zip(first, first[1:]))
    extent = end - first[0][0]                    # of one token's rows
    if rows and (T == 1 or extent <= st) and (b == 1 or extent + (T - 1) * st <= sb):
        return
    spans = sorted(_span(t) for t in grads)
    each = all(t[0, 0].numel() <= st or T == 1 for t in grads) and \
        all(t[0, 0].numel() + (T - 1) * st <= sb or b == 1 for t in grads)
    if not each or any(hi > lo for (_, hi), (lo, _) in zip(spans, spans[1:])):
        raise ValueError("dx, dB and dC must not share memory")


def _ssm_backward(handle, dev, code, dy, x, dt, A, B, C, D, dt_bias, h0, dhT, softplus, cu_seqlens, n, st, dxbc, ddt, dA,
                  dD, ddt_bias, dh0, workspace):
    b, T, H, P = x.shape
    G, N = B.shape[2:]
    ins = (dy, x, dt, A, B, C, D, dt_bias, h0, dhT, cu_seqlens)
    dx, dB, dC = dxbc
    if dx is None and dB is None and dC is None:
        # side by side, as the convolution that feeds the scan laid them out
        both = torch.empty(b, T, H * P + 2 * G * N, device=dev, dtype=x.dtype)
        dx, dB, dC = both.split((H * P, G * N, G * N), -1)
        dxbc = dx, dB, dC = dx.unflatten(-1, (H, P)), dB.unflatten(-1, (G, N)), dC.unflatten(-1, (G, N))
        grads = _strides(dx, "dx")
    else:
        if any(t is None for t in dxbc):
            raise ValueError("dx, dB and dC are given together or not at all")
        for t, name, like in ((dx, "dx", x), (dB, "dB", B), (dC, "dC", C)):
            _check(t, name, dev, like.shape, x.dtype, dense=False)
            _apart(t, name, *ins)
        grads = _strides(dx, "dx")
        # (one token has no stride to the next, one batch none to the next: _strides
        # gives a token's own width and 0 there)
        for t, name in ((dB, "dB"), (dC, "dC")):
            sb, stt = _strides(t, name)
            if t.numel() and (sb != grads[0] or (T > 1 and stt != grads[1])):
                raise ValueError("dx, dB and dC must have the same strides between batches and tokens")
        _side_by_side(dxbc, grads, b, T)
    ins += dxbc
    ddt = _out(ddt, "ddt", dev, (b, T, H), dt.dtype, ins)
    dA = _out(dA, "dA", dev, (H,), torch.float32, ins + (ddt,), A)
    dD = None if D is None else _out(dD, "dD", dev, (H,), torch.float32, ins + (ddt, dA), A)
    ddt_bias = None if dt_bias is None else _out(ddt_bias, "ddt_bias", dev, (H,), torch.float32, ins + (ddt, dA, dD), A)
    dh0 = None if h0 is None else _out(dh0, "dh0", dev, st, torch.float32, ins + (ddt, dA, dD, ddt_bias), h0)
    pr, need = _problem(SsmProblem, "gdn_workspace_bytes_ssm_backward", b, T, H, P, N, G, *_strides(x, "x"),
                        *_bc_strides(B, C), *_strides(dt, "dt"), *grads, n, code, _CODE[dt.dtype], softplus)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_ssm_backward", pr, dy.data_ptr(), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(h0),
          _ptr(cu_seqlens), _ptr(dhT), dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _ptr(dD), _ptr(ddt_bias),
          _ptr(dh0), _ptr(workspace), size, handle)
    return dx, ddt, dA, dB, dC, dD, ddt_bias, dh0


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, dt_softplus=True, slots=None, y=None, stream=None):
    """One token for each of b sequences: x [b, H, P], dt [b, H], B and C
    [b, G, N] (rows may be strided); state [S, H, N, P] fp32, moved on in place;
    slots as in conv_step.  Returns y [b, H, P]."""
    dev, code = _ssm_checks(x, dt, A, B, C, D, dt_bias, 1)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [S, H, N, P]")
    b, H, P = x.shape
    _check(state, "state", dev, (state.shape[0], H, B.shape[2], P), torch.float32)
    if slots is not None:
        _check(slots, "slots", dev, (b,), torch.int32)
    _apart(state, "state", x, dt, A, B, C, D, dt_bias, slots)
    return _on(dev, stream, _ssm_step, dev, code, x, dt, A, B, C, state, D, dt_bias, 1 if dt_softplus else 0, slots, y)


def _row_stride(t, name):
    """Between the rows of a step's input [b, ...] whose rows are dense."""
    if t.is_contiguous():
        return t.numel() // t.shape[0]
    want = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != want:
            raise ValueError("%s's rows must be contiguous" % name)
        want *= n
    return t.stride(0) if t.shape[0] != 1 else want


def _ssm_step(handle, dev, code, x, dt, A, B, C, state, D, dt_bias, softplus, slots, y):
    b, H, P = x.shape
    y = _out(y, "y", dev, x.shape, x.dtype, (x, dt, A, B, C, D, dt_bias, slots, state), x)
    if b:
        G, N = B.shape[1:]
        sb = _row_stride(B, "B")
        if _row_stride(C, "C") != sb:
            raise ValueError("B and C must have the same strides")
        pr, _ = _problem(SsmProblem, None, b, 1, H, P, N, G, _row_stride(x, "x"), H * P, sb, G * N, _row_stride(dt, "dt"), H,
                         0, 0, 0, code, _CODE[dt.dtype], softplus)
        _call("gdn_ssm_step", pr, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(dt_bias), state.data_ptr(),
              _ptr(slots), state.shape[0], y.data_ptr(), handle)
    return y
