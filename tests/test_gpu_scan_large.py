"""The selective scan's backward pass on tensors of more than 2^31 elements."""
import numpy as np
import pytest

from test_gpu_scan_backward import BF16, F32, TOL, off, reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_12_b200 import build

    build.build()


@pytest.mark.parametrize("D,zoh", [(16640, True), (16500, False)])
def test_past_32_bit_offsets(D, zoh):
    """b L D = 2.2e9, rows that start on 16 bytes and rows that do not; the
    second batch row's gradients of sampled channels, and dA of a channel with
    the first row's inputs."""
    import selective_state_space_12_b200 as ssd

    b, L, N = 2, 66000, 4
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.randn((b, L, D), generator=g, device="cuda", dtype=BF16) for _ in range(2))
    dt = torch.rand((b, L, D), generator=g, device="cuda", dtype=BF16).mul_(0.05).add_(0.01)
    A = -torch.exp(torch.rand((D, N), generator=g, device="cuda") * 2)
    B, C = (torch.randn((b, L, 1, N), generator=g, device="cuda", dtype=BF16) for _ in range(2))
    out = ssd.ssd_selective_scan_backward(x, dt, A, B, C, None, None, dy, zoh=zoh)
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    pick = [0, 8195, D - 1]
    cut = lambda t: t[:, :, pick].contiguous()
    s = dict(x=cut(x), dy=cut(dy), dt=cut(dt), A=A[pick].contiguous(), B=B, C=C, Dskip=None,
             bias=None, h0=None, dhf=None)
    ref = reference(s, zoh=zoh)
    for k in ("dx", "ddt"):
        assert off(out[k][1][:, pick].contiguous(), ref[k][1]) <= TOL, k
    assert off(out["dA"][pick], ref["dA"]) <= TOL
    assert off(out["dh0"][:, pick], ref["dh0"]) <= TOL
    assert np.isfinite(out["dB"].double().sum().item()) and np.isfinite(out["dC"].double().sum().item())
