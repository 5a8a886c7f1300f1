"""Binding of libgdn's layer operators (include/libgdn_layer.h): the
root-mean-square norm, layer norm, the short causal convolution, the selective
state space scan and the gated linear recurrence around the recurrence, and the
gated norm behind its heads.  As in the package itself every step runs in
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
    layer_norm_forward(x, weight, bias, residual) -> (y, s, scales)
    layer_norm_backward(dy, s, weight, bias, dres) -> (ds, dx, dweight, dbias)
    gate_norm_forward(x, z, weight, bias=None)    -> y
    gate_norm_backward(dy, x, z, weight, bias=None) -> (dx, dz, dweight, dbias)
    glr_forward(x, gate, h0=None)                 -> (y, hT)
    glr_backward(dy, x, gate, h0, dhT)            -> (dx, dgate, dbias, drate, dh0)
    glr_step(x, gate, state)                      -> y, the state in place

The work goes to ``stream``, or to the current stream of the tensors' device;
outputs and workspaces are allocated on that stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .layer_abi import (GDN_E4M3, LAYER_EXPORTS, ConvProblem, GateNormProblem, GlrProblem,  # noqa: F401
                        NormProblem, SsmProblem, declare)

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
# the bytes of workspace it needs.  (Fields are plain numbers: anything else would be
# found again by its identity, whatever it holds by then.)
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
    last = 1
    for n, s in zip(t.shape, t.stride()):
        last += (n - 1) * s
    return lo, lo + t.element_size() * last


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
    return _on(dev, stream, _norm_forward, dev, code, x, weight, residual, float(eps), out_dtype or dt, int(group), y, s, scales)


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
    return _on(dev, stream, _norm_backward, dev, code, dy, s, weight, dres, float(eps), ds, dx, dweight, workspace)


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
    if len(t.shape) == 2:
        n, D = t.shape
        s, one = t.stride()
        if one != 1 and D != 1:
            raise ValueError("%s's rows must be contiguous" % name)
        return s if n != 1 else D
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


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def layer_norm_forward(x, weight, bias=None, residual=None, *, eps=1e-5, out_dtype=None, group=0, y=None, s=None,
                       scales=None, stream=None):
    """s = x + residual (in the residual's type), y = (s - m) r w + b with m =
    mean(s) and r = 1 / sqrt(mean((s - m)^2) + eps) over the last dimension.

    Arguments and results as norm_forward's; bias [D] in the weight's type, or
    None (zero)."""
    dev = _device(x, "x")
    shape, dt = x.shape, x.dtype
    if x.dim() < 1 or shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1, got %s" % (tuple(shape),))
    code = _io_code(x, "x")
    _check(weight, "weight", dev, shape[-1:], dt, torch.float32)
    if bias is not None:
        _check(bias, "bias", dev, shape[-1:], weight.dtype)
    if residual is not None:
        _check(residual, "residual", dev, shape, dt, torch.float32)
    if out_dtype not in (None, dt, _FP8):
        raise TypeError("out_dtype must be %s or %s, got %s" % (dt, _FP8, out_dtype))
    if group not in (0, 128):
        raise ValueError("group must be 0 (a scale per row) or 128, got %r" % (group,))
    return _on(dev, stream, _layer_norm_forward, dev, code, x, weight, bias, residual, float(eps), out_dtype or dt, int(group), y, s, scales)


def _layer_norm_forward(handle, dev, code, x, weight, bias, residual, eps, od, group, y, s, scales):
    shape, D = x.shape, x.shape[-1]
    if x.is_contiguous():
        rows, stride = x.numel() // D, D
    else:
        merged = _rows(x)
        if merged is None:
            raise ValueError("x's rows must be contiguous and lie at one stride")
        rows, stride = merged
    y = _out(y, "y", dev, shape, od, (x, weight, bias, residual), x)
    scode = code
    if residual is not None:
        scode = _CODE[residual.dtype]
        if s is not None and s.data_ptr() == residual.data_ptr():
            _check(s, "s", dev, shape, residual.dtype)
            _apart(s, "s", x, weight, bias, y)
        else:
            s = _out(s, "s", dev, shape, residual.dtype, (x, weight, bias, residual, y), residual)
    else:
        _unwritten(s, "s", "a residual")
    if od is _FP8:
        scales = _out(scales, "scales", dev, shape[:-1] + ((D + group - 1) // group if group else 1,), torch.float32,
                      (x, weight, bias, residual, y, s))
    else:
        _unwritten(scales, "scales", "an 8-bit output")
    pr, _ = _problem(NormProblem, None, rows, D, stride, code, scode, _CODE[weight.dtype], _CODE[od], group, eps)
    _call("gdn_layer_norm_forward", pr, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), y.data_ptr(), _ptr(s), _ptr(scales),
          handle)
    return y, s, scales


def layer_norm_backward(dy, s, weight, bias=None, dres=None, *, eps=1e-5, x_dtype=None, ds=None, dx=None, dweight=None,
                        dbias=None, workspace=None, stream=None):
    """Layer norm's gradients: arguments as norm_backward's, and the forward's
    bias, whose values are not read.  Returns (ds, dx, dweight, dbias): dbias [D]
    fp32, None without a bias."""
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
    if bias is None:
        _unwritten(dbias, "dbias", "a bias")
    else:
        _check(bias, "bias", dev, shape[-1:], weight.dtype)
    if dres is not None:
        _check(dres, "dres", dev, shape, s.dtype)
    return _on(dev, stream, _layer_norm_backward, dev, code, dy, s, weight, bias, dres, float(eps), ds, dx, dweight, dbias, workspace)


def _layer_norm_backward(handle, dev, code, dy, s, weight, bias, dres, eps, ds, dx, dweight, dbias, workspace):
    shape, D = dy.shape, dy.shape[-1]
    ins = (dy, s, weight, bias)
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
    dbias = None if bias is None else _out(dbias, "dbias", dev, shape[-1:], torch.float32, ins + (dres, ds, dx, dweight))
    pr, need = _problem(NormProblem, "gdn_workspace_bytes_layer_norm_backward", dy.numel() // D, D, D, code, _CODE[s.dtype],
                        _CODE[weight.dtype], code, 0, eps)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_layer_norm_backward", pr, dy.data_ptr(), s.data_ptr(), weight.data_ptr(), _ptr(dres), ds.data_ptr(), _ptr(dx), dweight.data_ptr(),
          _ptr(dbias), _ptr(workspace), size, handle)
    return ds, ds if dx is None else dx, dweight, dbias


# ---------------------------------------------------------------------------
# gated norm
# ---------------------------------------------------------------------------

_ACT = {"silu": 0, "sigmoid": 1}


def _head_strides(shape, strides, name):
    """[..., H, D] as T tokens of H rows: (T, H, token stride, head stride).  Two
    dimensions are tokens of one row."""
    D = shape[-1]
    lead, H = (shape[:-2], shape[-2]) if len(shape) > 2 else (shape[:-1], 1)
    T = 1
    for n in lead:
        T *= n
    if T * H * D == 0:
        return T, H, H * D, D
    if D > 1 and strides[-1] != 1:
        raise ValueError("%s's rows must be contiguous" % name)
    st, want = H * D, None
    for n, s in zip(lead[::-1], strides[len(lead) - 1::-1] if lead else ()):
        if n == 1:
            continue
        if want is None:
            st = s
        elif s != want:
            raise ValueError("%s's tokens must lie at one stride" % name)
        want = s * n
    return T, H, st, strides[-2] if H > 1 else D


def _apart_rows(T, H, D, st, sh, name):
    """Rows of an output at two strides do not overlap."""
    if T * H < 2:
        return
    if H > 1 and sh < D or T > 1 and st < D:
        raise ValueError("%s's rows must not overlap" % name)
    if T > 1 and H > 1 and not (st >= (H - 1) * sh + D or sh >= (T - 1) * st + D):
        raise ValueError("%s's rows must not overlap" % name)


def _gate_norm_checks(x, z, weight, bias, activation, center):
    dev = _device(x, "x")
    code = _io_code(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1, got %s" % (tuple(x.shape),))
    _check(z, "z", dev, x.shape, x.dtype, dense=False)
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    each = weight.dim() == 2
    if each and x.dim() < 3:
        raise ValueError("a weight of its own for every head needs x of [..., H, D]")
    _check(weight, "weight", dev, x.shape[-2:] if each else x.shape[-1:], x.dtype, torch.float32)
    if bias is not None:
        if not center:
            raise ValueError("a bias needs center=True")
        _check(bias, "bias", dev, weight.shape, weight.dtype)
    if activation not in _ACT:
        raise ValueError("activation must be 'silu' or 'sigmoid', got %r" % (activation,))
    return dev, code, each


@functools.lru_cache(maxsize=4096)
def _gate_norm_problem(size_of, shape, xs, zs, dzs, code, wcode, each, first, center, act, eps):
    T, H, xt, xh = _head_strides(shape, xs, "x")
    _, _, zt, zh = _head_strides(shape, zs, "z")
    dt, dh = 0, 0
    if dzs is not None:
        _, _, dt, dh = _head_strides(shape, dzs, "dz")
        _apart_rows(T, H, shape[-1], dt, dh, "dz")
    return _problem(GateNormProblem, size_of, T, H, shape[-1], xt, xh, zt, zh, dt, dh, code, wcode, int(each), int(first), int(center),
                    act, eps)


def gate_norm_forward(x, z, weight, bias=None, *, eps=1e-5, activation="silu", gate_first=False, center=False, y=None,
                      stream=None):
    """The norm behind a recurrence's heads: y = n(x) act(z), or with gate_first
    y = n(x act(z)); n(v) = v r w with r = 1 / sqrt(mean(v^2) + eps) over the last
    dimension, and centred (v - m) r w + b.

    x and z [..., H, D] (or [..., D]) bf16 or fp32, whose tokens and heads may each
    lie at a stride; weight [D], or [H, D] for weights of each head, in x's type or
    fp32; bias like it (with center), or None.  activation: "silu" or "sigmoid".
    Returns y, dense."""
    dev, code, each = _gate_norm_checks(x, z, weight, bias, activation, center)
    return _on(dev, stream, _gate_norm_forward, dev, code, x, z, weight, bias, each, bool(gate_first), bool(center), _ACT[activation],
               float(eps), y)


def _gate_norm_forward(handle, dev, code, x, z, weight, bias, each, first, center, act, eps, y):
    y = _out(y, "y", dev, x.shape, x.dtype, (x, z, weight, bias), x)
    pr, _ = _gate_norm_problem(None, x.shape, x.stride(), z.stride(), None, code, _CODE[weight.dtype], each, first, center, act, eps)
    _call("gdn_gate_norm_forward", pr, x.data_ptr(), z.data_ptr(), weight.data_ptr(), _ptr(bias), y.data_ptr(), handle)
    return y


def gate_norm_backward(dy, x, z, weight, bias=None, *, eps=1e-5, activation="silu", gate_first=False, center=False, dx=None,
                       dz=None, dweight=None, dbias=None, workspace=None, stream=None):
    """The gated norm's gradients for dy (dense, like x).  Returns (dx, dz, dweight,
    dbias): dx dense; dz may be given as a part of a wider buffer, as z is of a
    projection's rows; dweight and dbias fp32 like the weight and the bias (None
    without one)."""
    dev, code, each = _gate_norm_checks(x, z, weight, bias, activation, center)
    _check(dy, "dy", dev, x.shape, x.dtype)
    if bias is None:
        _unwritten(dbias, "dbias", "a bias")
    return _on(dev, stream, _gate_norm_backward, dev, code, dy, x, z, weight, bias, each, bool(gate_first), bool(center), _ACT[activation],
               float(eps), dx, dz, dweight, dbias, workspace)


def _gate_norm_backward(handle, dev, code, dy, x, z, weight, bias, each, first, center, act, eps, dx, dz, dweight, dbias, workspace):
    ins = (dy, x, z, weight, bias)
    dx = _out(dx, "dx", dev, x.shape, x.dtype, ins, x)
    if dz is None:
        dz = _out(None, "dz", dev, x.shape, x.dtype, ins, x)
    else:
        _check(dz, "dz", dev, x.shape, x.dtype, dense=False)
        _apart(dz, "dz", *ins, dx)
    dweight = _out(dweight, "dweight", dev, weight.shape, torch.float32, ins + (dx, dz), weight)
    dbias = None if bias is None else _out(dbias, "dbias", dev, bias.shape, torch.float32, ins + (dx, dz, dweight), bias)
    pr, need = _gate_norm_problem("gdn_workspace_bytes_gate_norm_backward", x.shape, x.stride(), z.stride(), dz.stride(), code,
                                  _CODE[weight.dtype], each, first, center, act, eps)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_gate_norm_backward", pr, dy.data_ptr(), x.data_ptr(), z.data_ptr(), weight.data_ptr(), _ptr(bias), dx.data_ptr(), dz.data_ptr(),
          dweight.data_ptr(), _ptr(dbias), _ptr(workspace), size, handle)
    return dx, dz, dweight, dbias


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------

_FORM = {"log": 0, "sigmoid": 1, "rate": 2}
_SCALE = {None: 0, "complement": 1, "norm": 2}


def _glr_checks(x, gate, gate_bias, rate, form, scale, dims):
    dev = _device(x, "x")
    code = _io_code(x, "x")
    if x.dim() != dims or x.shape[-1] < 1:
        raise ValueError("x must be %s, got %s" % ("[B, T, D]" if dims == 3 else "[B, D]", tuple(x.shape)))
    _check(gate, "gate", dev, x.shape, x.dtype, torch.float32, dense=False)
    if form not in _FORM:
        raise ValueError("form must be 'log', 'sigmoid' or 'rate', got %r" % (form,))
    if scale not in _SCALE:
        raise ValueError("scale must be None, 'complement' or 'norm', got %r" % (scale,))
    if (form == "rate") != (rate is not None):
        raise ValueError("a rate is needed for form 'rate'" if rate is None else "a rate is for form 'rate' only")
    if gate_bias is not None:
        _check(gate_bias, "gate_bias", dev, x.shape[-1:], torch.float32)
    if rate is not None:
        _check(rate, "rate", dev, x.shape[-1:], torch.float32)
    return dev, code


def _token_strides(shape, strides, name):
    """(batch, token) strides of [B, T, D] whose rows are dense (see _strides)."""
    B, T, D = shape
    if strides[2] != 1 and D != 1 and B * T * D:
        raise ValueError("%s must be contiguous behind its token dimension" % name)
    return (strides[0] if B != 1 else 0), (strides[1] if T != 1 else D)


@functools.lru_cache(maxsize=4096)
def _glr_problem(size_of, shape, xs, gs, grads, n, code, gcode, form, scale):
    """grads: the strides of dy, dx and dgate, or None."""
    at = _token_strides(shape, xs, "x") + _token_strides(shape, gs, "gate")
    for name, strides in zip(("dy", "dx", "dgate"), grads or ()):
        at += _token_strides(shape, strides, name)
    at += (0, 0) * (0 if grads else 3)
    return _problem(GlrProblem, size_of, *shape, *at, n, code, gcode, form, scale)


def glr_forward(x, gate, h0=None, *, gate_bias=None, rate=None, form="log", scale=None, cu_seqlens=None, y=None, hT=None,
                output_final_state=True, workspace=None, stream=None):
    """Gated linear recurrence per channel: h_t = a_t h_{t-1} + c_t x_t, y_t = h_t.

    form: with v = gate + gate_bias, "log": log a = v; "sigmoid": a = sigmoid(v);
    "rate": log a = -rate sigmoid(v).  scale: c = 1 (None), 1 - a ("complement") or
    sqrt(1 - a^2) ("norm").  x [B, T, D] bf16 or fp32, gate like it in x's type or
    fp32 (tokens of each may be strided); gate_bias, rate [D] fp32; h0 [B, D] fp32, or
    [n, D] with cu_seqlens (as in conv_forward).  Returns (y [B, T, D], hT like h0
    or None)."""
    dev, code = _glr_checks(x, gate, gate_bias, rate, form, scale, 3)
    n = _packed(cu_seqlens, dev, x.shape[0])
    if h0 is not None:
        _check(h0, "h0", dev, (n or x.shape[0], x.shape[2]), torch.float32)
    return _on(dev, stream, _glr_forward, dev, code, x, gate, h0, gate_bias, rate, _FORM[form], _SCALE[scale], cu_seqlens, n, y, hT,
               output_final_state, workspace)


def _glr_forward(handle, dev, code, x, gate, h0, gate_bias, rate, form, scale, cu_seqlens, n, y, hT, want, workspace):
    B, T, D = x.shape
    ins = (x, gate, h0, gate_bias, rate, cu_seqlens)
    y = _out(y, "y", dev, x.shape, x.dtype, ins, x)
    if hT is not None or want:
        hT = _out(hT, "hT", dev, (n or B, D), torch.float32, ins + (y,), h0)
    pr, need = _glr_problem("gdn_workspace_bytes_glr", x.shape, x.stride(), gate.stride(), None, n, code, _CODE[gate.dtype], form, scale)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_glr_forward", pr, x.data_ptr(), gate.data_ptr(), _ptr(gate_bias), _ptr(rate), _ptr(h0), _ptr(cu_seqlens), y.data_ptr(),
          _ptr(hT), _ptr(workspace), size, handle)
    return y, hT


def glr_backward(dy, x, gate, h0=None, dhT=None, *, gate_bias=None, rate=None, form="log", scale=None, cu_seqlens=None,
                 dx=None, dgate=None, dbias=None, drate=None, dh0=None, workspace=None, stream=None):
    """The recurrence's gradients for dy [B, T, D] (tokens may be strided) and dhT
    (of the final states, or None); the states are formed again from the inputs.
    Returns (dx, dgate, dbias, drate, dh0): dx in x's type, dgate in the gate's, dbias
    (of gate_bias), drate and dh0 fp32, None where gate_bias, rate and h0 are.  dx and
    dgate may be given as parts of one buffer, as the gradient of the projection
    that x and the gate come from."""
    dev, code = _glr_checks(x, gate, gate_bias, rate, form, scale, 3)
    n = _packed(cu_seqlens, dev, x.shape[0])
    _check(dy, "dy", dev, x.shape, x.dtype, dense=False)
    if gate_bias is None:
        _unwritten(dbias, "dbias", "a gate_bias")
    if rate is None:
        _unwritten(drate, "drate", "a rate")
    if h0 is None:
        _unwritten(dh0, "dh0", "an h0")
    for t, name in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _check(t, name, dev, (n or x.shape[0], x.shape[2]), torch.float32)
    return _on(dev, stream, _glr_backward, dev, code, dy, x, gate, h0, dhT, gate_bias, rate, _FORM[form], _SCALE[scale], cu_seqlens, n,
               dx, dgate, dbias, drate, dh0, workspace)


def _token_rows_apart(dx, dgate):
    """dx and dgate, each [B, T, D] at strides of its own, hold no element twice."""
    B, T, D = dx.shape
    if not dx.numel():
        return
    at, to = _strides(dx, "dx"), _strides(dgate, "dgate")
    _apart_rows(T, B, D, at[1], at[0], "dx")
    _apart_rows(T, B, D, to[1], to[0], "dgate")
    (a, a1), (b, b1) = _span(dx), _span(dgate)
    if a1 <= b or b1 <= a:
        return
    # parts of one buffer: rows at the same strides, of which no two are nearer than D
    apart, off = divmod(b - a, dx.element_size())
    if dx.dtype is dgate.dtype and at == to and not off:
        (so, no), (si, ni) = sorted(((at[0], B), (at[1], T)), reverse=True)
        near = lambda d, s, n: {max(1 - n, min(n - 1, -d // s + k)) for k in (-1, 0, 1, 2)} if n > 1 else {0}  # noqa: E731
        if all(abs(apart + o * so + i * si) >= D for o in near(apart, so, no) for i in near(apart + o * so, si, ni)):
            return
    raise ValueError("dx and dgate must not share memory")


def _glr_backward(handle, dev, code, dy, x, gate, h0, dhT, gate_bias, rate, form, scale, cu_seqlens, n, dx, dgate, dbias, drate, dh0,
                  workspace):
    B, T, D = x.shape
    ins = (dy, x, gate, h0, dhT, gate_bias, rate, cu_seqlens)
    if dx is None and dgate is None:
        dx = torch.empty(B, T, D, device=dev, dtype=x.dtype)
        dgate = torch.empty(B, T, D, device=dev, dtype=gate.dtype)
    else:
        for t, name, like in ((dx, "dx", x), (dgate, "dgate", gate)):
            if t is not None:
                _check(t, name, dev, x.shape, like.dtype, dense=False)
                _apart(t, name, *ins)
        dx = torch.empty(B, T, D, device=dev, dtype=x.dtype) if dx is None else dx
        dgate = torch.empty(B, T, D, device=dev, dtype=gate.dtype) if dgate is None else dgate
        _token_rows_apart(dx, dgate)
    ins += (dx, dgate)
    dbias = None if gate_bias is None else _out(dbias, "dbias", dev, (D,), torch.float32, ins, gate_bias)
    drate = None if rate is None else _out(drate, "drate", dev, (D,), torch.float32, ins + (dbias,), rate)
    dh0 = None if h0 is None else _out(dh0, "dh0", dev, h0.shape, torch.float32, ins + (dbias, drate), h0)
    pr, need = _glr_problem("gdn_workspace_bytes_glr_backward", x.shape, x.stride(), gate.stride(), (dy.stride(), dx.stride(), dgate.stride()),
                            n, code, _CODE[gate.dtype], form, scale)
    workspace, size = _workspace(need, dev, workspace)
    _call("gdn_glr_backward", pr, dy.data_ptr(), x.data_ptr(), gate.data_ptr(), _ptr(gate_bias), _ptr(rate), _ptr(h0), _ptr(cu_seqlens),
          _ptr(dhT), dx.data_ptr(), dgate.data_ptr(), _ptr(dbias), _ptr(drate), _ptr(dh0), _ptr(workspace), size, handle)
    return dx, dgate, dbias, drate, dh0


def glr_step(x, gate, state, *, gate_bias=None, rate=None, form="log", scale=None, slots=None, y=None, stream=None):
    """One token for each of B sequences: x and gate [B, D] (rows may be strided);
    state [S, D] fp32, moved on in place; slots as in conv_step; the rest as in
    glr_forward.  Returns y [B, D]."""
    dev, code = _glr_checks(x, gate, gate_bias, rate, form, scale, 2)
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be [S, D]")
    B, D = x.shape
    _check(state, "state", dev, (state.shape[0], D), torch.float32)
    if slots is not None:
        _check(slots, "slots", dev, (B,), torch.int32)
    _apart(state, "state", x, gate, gate_bias, rate, slots)
    return _on(dev, stream, _glr_step, dev, code, x, gate, state, gate_bias, rate, _FORM[form], _SCALE[scale], slots, y)


@functools.lru_cache(maxsize=4096)
def _glr_step_problem(B, D, xs, gs, code, gcode, form, scale):
    return ctypes.byref(GlrProblem(B, 1, D, xs, D, gs, D, 0, 0, 0, 0, 0, 0, 0, code, gcode, form, scale))


def _glr_step(handle, dev, code, x, gate, state, gate_bias, rate, form, scale, slots, y):
    B, D = x.shape
    y = _out(y, "y", dev, x.shape, x.dtype, (x, gate, gate_bias, rate, slots, state), x)
    if B:
        pr = _glr_step_problem(B, D, _row_stride(x, "x"), _row_stride(gate, "gate"), code, _CODE[gate.dtype], form, scale)
        _call("gdn_glr_step", pr, x.data_ptr(), gate.data_ptr(), _ptr(gate_bias), _ptr(rate), state.data_ptr(), _ptr(slots), state.shape[0],
              y.data_ptr(), handle)
    return y
