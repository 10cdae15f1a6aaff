"""A call with stream= takes its scratch and outputs from that stream's memory
(no GPU needed: torch's streams are stood in for)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
import selective_state_space_12_b200 as ssd
from selective_state_space_12_b200 import ssd as binding


class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


CALLER, OWN, OTHER_GPU = Stream(1), Stream(2), Stream(3, 1)


@pytest.fixture
def now(monkeypatch):
    from selective_state_space_12_b200 import build

    build.build()
    at = [CALLER]

    @contextlib.contextmanager
    def stream(s):
        at.append(s)
        try:
            yield
        finally:
            at.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[-1])
    monkeypatch.setattr(torch.cuda, "set_stream", lambda s: at.__setitem__(-1, s))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(binding, "_current_handle", lambda device: at[-1].cuda_stream)
    return at


def test_scratch_comes_from_the_calls_stream(now, monkeypatch):
    taken = []
    monkeypatch.setattr(binding, "_workspace", lambda *a: taken.append(now[-1]) or (None, 0))
    x, lam, h = torch.zeros((1, 8, 4)), torch.zeros(4), torch.zeros((1, 1, 4))
    A, B = -torch.ones((4, 16)), torch.zeros((1, 8, 1, 16))
    ck = ssd.GatedCheckpoint8(1, 8, 4, device="cpu")
    calls = [lambda s: ssd.ssd_gated_scan(x, x, x, lam, stream=s),
             lambda s: ssd.ssd_gated_scan_backward(x, x, x, lam, h, x, stream=s),
             lambda s: ssd.ssd_gated_scan_backward_ckpt8(ck, lam, x, stream=s),
             lambda s: ssd.ssd_selective_scan_backward(x, x, A, B, B, None, None, x, stream=s)]
    for call in calls:
        for s, want in ((OWN, OWN), (CALLER, CALLER), (None, CALLER), (OTHER_GPU, OTHER_GPU)):
            with pytest.raises(ValueError, match="CUDA"):  # the tensors are not on a GPU
                call(s)
            assert taken.pop() is want and now == [CALLER]


def test_tensors_are_kept_for_both_streams(now, monkeypatch):
    kept = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s)))
    x, y = torch.zeros(4), torch.zeros(4)
    ck = ssd.GatedCheckpoint8(1, 8, 4, device="cpu")
    for out in (y, (y, None), dict(dx=y, dh0=None)):
        inside = []

        def fn(x, ck, c, stream):
            inside.append(now[-1])
            return out

        assert binding._on_stream(fn, dict(x=x, ck=ck, c=8.0, stream=OWN)) is out
        assert inside == [OWN]
        want = [(t.data_ptr(), OWN) for t in (x, ck.q, ck.e, ck.states)] + [(y.data_ptr(), CALLER)]
        assert kept == want
        kept.clear()
