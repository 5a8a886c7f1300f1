"""The layer operators' binding on the CPU: what it hands to the library, and
what it refuses before that.  Calls are caught at the library's door, with CPU
tensors in the place of the device's."""
import os
import subprocess
import sys
import types

import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer as L

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library: (name, problem, arguments)."""
    seen = []
    monkeypatch.setattr(L, "_device", lambda t, name: t.device)
    monkeypatch.setattr(L, "_on", lambda device, stream, work, *args: work(None, *args))
    monkeypatch.setattr(L, "_call", lambda name, pr, *args: seen.append((name, pr._obj, args)))
    return seen


def scan(b, T, H=4, P=64, N=64, G=1, dt=BF):
    d = types.SimpleNamespace(
        x=torch.zeros(b, T, H, P, dtype=dt), dt=torch.zeros(b, T, H, dtype=dt), A=-torch.ones(H),
        B=torch.zeros(b, T, G, N, dtype=dt), C=torch.zeros(b, T, G, N, dtype=dt), dy=torch.zeros(b, T, H, P, dtype=dt))
    d.args = (d.dy, d.x, d.dt, d.A, d.B, d.C)
    return d


def side_by_side(b, T, H, P, G, N, dt=BF, first=0):
    buf = torch.zeros(b, T, first + H * P + 2 * G * N, dtype=dt)[..., first:]
    dx, dB, dC = buf.split((H * P, G * N, G * N), -1)
    return dict(dx=dx.unflatten(-1, (H, P)), dB=dB.unflatten(-1, (G, N)), dC=dC.unflatten(-1, (G, N)))


@pytest.mark.parametrize("b,H,P,N,G", [(2, 4, 64, 64, 1), (4, 8, 64, 64, 1), (3, 1, 64, 128, 1), (2, 2, 128, 64, 2)])
def test_scan_gradients_of_single_tokens_have_one_batch_stride(calls, b, H, P, N, G):
    """The library takes one stride between batches for dx, dB and dC, also where
    every batch is a single token."""
    d = scan(b, 1, H, P, N, G)
    own = dict(dx=torch.zeros_like(d.x), dB=torch.zeros_like(d.B), dC=torch.zeros_like(d.C))
    if H * P != G * N:
        with pytest.raises(ValueError, match="same strides"):
            gdn.ssm_backward(*d.args, **own)
        assert not calls
    one = side_by_side(b, 1, H, P, G, N)
    got = gdn.ssm_backward(*d.args, **one)
    assert got[0] is one["dx"] and got[3] is one["dB"] and got[4] is one["dC"]
    (name, pr, args), = calls
    assert name == "gdn_ssm_backward" and pr.dxbc_stride_b == H * P + 2 * G * N
    # batches of one buffer that overlap
    wide = torch.zeros(2 * b * H * P + 8 * b * G * N, dtype=BF)
    near = dict(dx=wide.as_strided((b, 1, H, P), (8, H * P, P, 1)), dB=wide[H * P:].as_strided((b, 1, G, N), (8, G * N, N, 1)),
                dC=wide[H * P + G * N:].as_strided((b, 1, G, N), (8, G * N, N, 1)))
    with pytest.raises(ValueError, match="share memory"):
        gdn.ssm_backward(*d.args, **near)
    assert len(calls) == 1


def test_scan_gradients_of_one_batch_or_no_tokens_need_no_common_stride(calls):
    for b, T in ((1, 1), (3, 0)):
        d = scan(b, T)
        gdn.ssm_backward(*d.args, dx=torch.zeros_like(d.x), dB=torch.zeros_like(d.B), dC=torch.zeros_like(d.C))
    assert len(calls) == 2


def test_the_library_loads_without_torch():
    """As the rest of the package: torch is imported where tensors are worked on."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import chunked_gated_delta_prepare_amd as gdn\n"
            "lib = gdn.load_library()\n"
            "assert lib.gdn_ssm_forward.argtypes and lib.gdn_workspace_bytes_ssm.restype\n")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0, run.stderr


def test_the_steps_states_share_memory_with_no_input(calls):
    """A state is written in place while other rows and heads still read the inputs."""
    B, D, W, S = 3, 64, 4, 5
    pool = torch.zeros(S, W - 1, D)
    at = lambda *shape, first=0: pool.view(-1)[first:first + torch.Size(shape).numel()].view(*shape)  # noqa: E731
    x, w, b = torch.zeros(B, D), torch.zeros(D, W), torch.zeros(D)
    slots = torch.zeros(B, dtype=torch.int32)
    gdn.conv_step(x, pool, w, b, slots=slots)
    for kw in (dict(x=at(B, D)), dict(weight=at(D, W, first=7)), dict(bias=at(D, first=S * (W - 1) * D - D)),
               dict(slots=pool.view(torch.int32).view(-1)[:B])):
        with pytest.raises(ValueError, match="share memory"):
            gdn.conv_step(**{**dict(x=x, state=pool, weight=w, bias=b, slots=slots), **kw})
    H, P, N, G = 2, 64, 64, 1
    pool = torch.zeros(S, H, N, P)
    d = dict(x=torch.zeros(B, H, P), dt=torch.zeros(B, H), A=-torch.ones(H), B=torch.zeros(B, G, N), C=torch.zeros(B, G, N),
             D=torch.ones(H), dt_bias=torch.zeros(H), slots=slots)
    gdn.ssm_step(**d, state=pool)
    for k in d:
        inside = (pool.view(torch.int32) if k == "slots" else pool).view(-1)[64:64 + d[k].numel()].view(d[k].shape)
        with pytest.raises(ValueError, match="share memory"):
            gdn.ssm_step(**{**d, k: inside}, state=pool)
    assert [c[0] for c in calls] == ["gdn_conv_step", "gdn_ssm_step"]


def test_outputs_that_would_not_be_written_are_refused(calls):
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="residual"):
        gdn.norm_forward(x, w, s=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="scales"):
        gdn.norm_forward(x, w, scales=torch.zeros(4, 1))
    taps, tokens = torch.zeros(64, 4), torch.zeros(1, 7, 64)
    with pytest.raises(ValueError, match="dbias"):
        gdn.conv_backward(tokens, tokens, taps, dbias=torch.zeros(64))
    with pytest.raises(ValueError, match="dinitial"):
        gdn.conv_backward(tokens, tokens, taps, dinitial=torch.zeros(1, 3, 64))
    d = scan(1, 5)
    for name, shape in (("dD", (4,)), ("ddt_bias", (4,)), ("dh0", (1, 4, 64, 64))):
        with pytest.raises(ValueError, match=name):
            gdn.ssm_backward(*d.args, **{name: torch.zeros(shape)})
    assert not calls
