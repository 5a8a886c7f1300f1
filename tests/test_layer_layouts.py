"""Where gradients may be written: every layout whose elements are all apart is taken, every
other is refused (CPU tensors; calls are caught at the library's door)."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer as L


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(L, "_device", lambda t, name: t.device)
    monkeypatch.setattr(L, "_on", lambda device, stream, work, *args: work(None, *args))
    monkeypatch.setattr(L, "_call", lambda name, pr, *args: seen.append((name, pr._obj, args)))
    return seen


def test_glr_gradients_in_any_layout_of_one_buffer(calls):
    B, T, D = 3, 7, 64
    x, gate = torch.zeros(B, T, D), torch.zeros(B, T, D)
    wide, per_batch, time_major = torch.zeros(B, T, 2 * D + 5), torch.zeros(B, 2, T, D), torch.zeros(T, B, 2 * D)
    ways = [(wide[..., :D], wide[..., D:2 * D]), (per_batch[:, 0], per_batch[:, 1]), (per_batch[:, 1], per_batch[:, 0]),
            (time_major[..., D:].transpose(0, 1), time_major[..., :D].transpose(0, 1)),
            (torch.zeros(T, B, D).transpose(0, 1), torch.zeros(B, T, D)), (torch.zeros(T, B, D).transpose(0, 1), None),
            (torch.zeros(2, T, B, D)[0].transpose(0, 1), torch.zeros(2, T, B, D)[1].transpose(0, 1))]
    alternate = torch.zeros(T, 2, B, D)           # a token's rows of dx, then of dgate
    ways.append((alternate[:, 0].transpose(0, 1), alternate[:, 1].transpose(0, 1)))
    for dx, dg in ways:
        out = gdn.glr_backward(x, x, gate, dx=dx, dgate=dg)
        assert out[0] is dx and (dg is None or out[1] is dg)
        pr = calls[-1][1]
        assert (pr.dx_stride_b, pr.dx_stride_t) == dx.stride()[:2]
    assert len(calls) == len(ways)


def test_glr_gradients_that_share_an_element_are_refused(calls):
    """Against a count of the elements, for strides and distances around those that fit."""
    B, T, D = 2, 3, 4
    x, gate = torch.zeros(B, T, D), torch.zeros(B, T, D)
    taken = refused = 0
    for sb, st in ((12, 4), (13, 4), (4, 8), (5, 9), (24, 8), (11, 4), (3, 20), (26, 9), (12, 3), (4, 7)):
        for apart in itertools.chain(range(0, 40), (-4, -3, -8, -12)):
            buf = torch.zeros(120)
            dx, dg = (buf.as_strided((B, T, D), (sb, st, 1), at) for at in (20, 20 + apart))
            places = [i for t in (dx, dg) for i in
                      (t.storage_offset() + b * sb + k * st + d for b in range(B) for k in range(T) for d in range(D))]
            before = len(calls)
            if len(set(places)) == len(places):
                gdn.glr_backward(x, x, gate, dx=dx, dgate=dg)
                taken += 1
            else:
                with pytest.raises(ValueError, match="overlap|share"):
                    gdn.glr_backward(x, x, gate, dx=dx, dgate=dg)
                refused += 1
            assert (len(calls) > before) == (len(set(places)) == len(places)), (sb, st, apart)
    assert taken > 50 and refused > 50
