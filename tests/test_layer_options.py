"""Options given as numbers of other kinds than Python's own: problems are cached by their
values, so a tensor or an array must count with what it holds at the call (CPU tensors; calls are
caught at the library's door)."""
import pytest

torch = pytest.importorskip("torch")
np = pytest.importorskip("numpy")

import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer as L


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(L, "_device", lambda t, name: t.device)
    monkeypatch.setattr(L, "_on", lambda device, stream, work, *args: work(None, *args))
    monkeypatch.setattr(L, "_call", lambda name, pr, *args: seen.append((name, pr._obj, args)))
    return seen


@pytest.mark.parametrize("make", [lambda v: torch.tensor(v), lambda v: np.array(v, dtype=np.float32)])
def test_eps_counts_with_its_value_at_the_call(calls, make):
    x, w = torch.zeros(4, 64), torch.ones(64)
    for f in (lambda e: gdn.norm_forward(x, w, eps=e), lambda e: gdn.norm_backward(x, x, w, eps=e),
              lambda e: gdn.layer_norm_forward(x, w, eps=e), lambda e: gdn.layer_norm_backward(x, x, w, eps=e),
              lambda e: gdn.gate_norm_forward(x, x, w, eps=e), lambda e: gdn.gate_norm_backward(x, x, x, w, eps=e)):
        eps = make(0.25)
        f(eps)
        eps[...] = 0.5
        f(eps)
        assert [c[1].eps for c in calls[-2:]] == [0.25, 0.5]


def test_flags_count_with_their_value_at_the_call(calls):
    x, w, flag = torch.zeros(4, 64), torch.ones(64), torch.tensor(False)
    for name in ("gate_first", "center"):
        for f in (lambda: gdn.gate_norm_forward(x, x, w, **{name: flag}), lambda: gdn.gate_norm_backward(x, x, x, w, **{name: flag})):
            flag.fill_(False)
            f()
            flag.fill_(True)
            f()
            assert [getattr(c[1], name) for c in calls[-2:]] == [0, 1]


def test_groups_count_with_their_value_at_the_call(calls):
    x, w, group = torch.zeros(4, 256), torch.ones(256), torch.tensor(0)
    for f in (gdn.norm_forward, gdn.layer_norm_forward):
        for n in (0, 128):
            group.fill_(n)
            f(x, w, out_dtype=torch.float8_e4m3fn, group=group)
        assert [c[1].group for c in calls[-2:]] == [0, 128]
