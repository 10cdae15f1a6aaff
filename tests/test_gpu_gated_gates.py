"""Gates at their ends in the gated recurrence, against the definition in 64
bits channel by channel: an output's error, less its rounding, is a share of the
larger of the value and its channel's rms, so that no channel hides behind
another. The bound is the one of the recurrence's other tests."""
import numpy as np
import pytest

from test_gpu_gated import TOL, make, reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_12_b200 import build

    build.build()


def off_by_channel(got, ref, of=None):
    """(b, L, D); a share of the channel's own rms (of ``of``: a last state by
    itself may be as small as the terms that make it happen to cancel)."""
    of = ref if of is None else of
    half = torch.finfo(got.dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    axes = tuple(range(of.ndim - 1))
    size = np.maximum(np.abs(ref), np.sqrt(np.mean(np.square(of), axis=axes)))
    gap = np.maximum(np.abs(got - ref) - half * np.abs(ref), 0)
    return float(np.max(np.where(gap > 0, gap / np.maximum(size, 1e-300), 0)))


def both(s, **kw):
    import selective_state_space_12_b200 as ssd

    b, L, D = s["x"].shape
    st = torch.empty((b, ssd.gated_blocks(L), D), device="cuda")
    y, hf = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                               states=st)
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"],
                                    reset=s["reset"])
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    return y, hf, g


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shut", [float("-inf"), -3e38, -1e4, -200.0])
@pytest.mark.parametrize("D", [40, 5130])
def test_a_shut_decay_gate_holds_the_state(D, shut, dtype):
    """sigmoid(r) = 0 (below 2^-126 at the least): a = 1 and m = 0, so a masked
    stretch of any length leaves the state as it was and passes the gradient
    through; a sequence that is masked from its start on stays 0. To the bit from
    the block after the one that the stretch begins in: there the state is carried
    on by the map of several tokens, rounded otherwise than token by token."""
    import selective_state_space_12_b200 as ssd

    L, a, b = 3000, 70, 2900  # masked from a to b
    s = make(2, L, D, dtype=dtype, seed=5)
    s["x"][:, a:b] = 50.0
    s["r"][:, a:b] = shut
    s["h0"][1], s["r"][1, :a] = 0.0, shut
    y, hf, g = both(s)
    assert torch.equal(y[0, 128:b], y[0, 128:129].expand(b - 128, D))
    # half a step for each of the two where they are rounded, the bound for how they are reached
    gap = (y[0, 128].double() - y[0, a - 1].double()).abs()
    size = y[0, a - 1].double().abs().clamp(min=float(y[0, :a].double().square().mean().sqrt()))
    assert float((gap / size).max()) <= TOL + torch.finfo(dtype).eps
    assert not y[1, :b].any()
    for k in ("dx", "dr", "di"):
        assert not g[k][:, a:b].any(), k
    h = s["h0"].clone()
    for t in (a, a + 1):
        y1 = ssd.ssd_gated_step(h, *(s[k][:, t].contiguous() for k in ("x", "r", "i")), s["lam"])
    assert torch.equal(h, s["h0"]) and torch.equal(y1, s["h0"].to(dtype))


@pytest.mark.parametrize("D", [40, 5130])
def test_gates_that_are_all_but_shut(D):
    """r and i from -70 to -40, below 2^-63 in part: m and sigmoid(i) keep their
    bits, from a zero state."""
    s = make(1, 130, D, h0=False, seed=6)
    s["r"] = s["r"] * 0 - torch.linspace(40, 70, D, device="cuda")
    y, hf, g = both(s)
    ref, grads = reference(s["x"], s["r"], s["i"], s["lam"], None, None, s["dy"], None)
    assert off_by_channel(y, ref) <= TOL and off_by_channel(hf, ref[:, -1], ref) <= TOL
    for k in ("dx", "di", "dr"):
        assert off_by_channel(g[k], grads[k]) <= TOL, k
    s = make(1, 130, D, h0=False, seed=7)
    s["i"] = s["i"] * 0 - torch.linspace(40, 70, D, device="cuda")
    y, hf, g = both(s)
    ref, grads = reference(s["x"], s["r"], s["i"], s["lam"], None, None, s["dy"], None)
    assert off_by_channel(y, ref) <= TOL
    for k in ("dx", "di"):
        assert off_by_channel(g[k], grads[k]) <= TOL, k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [10, 64])
def test_a_reset_tokens_decay_gate_counts_for_nothing(D, dtype):
    """Whatever r holds at a reset, NaN and infinities too."""
    s = make(3, 200, D, dtype=dtype, seed=8)
    reset = torch.zeros((3, 200), dtype=torch.uint8, device="cuda")
    reset[0, 17] = reset[1, 64] = reset[2, 199] = reset[0, 128] = 1
    s["reset"] = reset
    y, hf, g = both(s)
    for v in (float("nan"), float("inf"), float("-inf")):
        s["r"][reset != 0] = v
        y2, hf2, g2 = both(s)
        assert torch.equal(y, y2) and torch.equal(hf, hf2)
        for k in g:
            assert torch.equal(g[k], g2[k]), k
    assert not g["dr"][reset != 0].any()


def fast_tolerance(lam):
    """The bound, and for a = exp(-q) what an error of q makes of it: q is within
    about 5e-7 of its value (c softplus(lam) 2e-7, its gate 2e-7, their product
    and the exponent's rounding 1e-7), so a within 5e-7 q, q <= c softplus(lam)."""
    return TOL + 5e-7 * 8.0 * float(np.log1p(np.exp(lam)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [40, 96, 5130])
@pytest.mark.parametrize("lam", [0.0, 2.0, 4.0])
def test_channels_that_forget_fast(lam, D, dtype):
    """Decays of e^-3 to e^-32 a token in every channel: the gradients of the
    decay gate and of lam, which are in proportion to them, keep their bits."""
    s = make(2, 150, D, dtype=dtype, reset=True, seed=9)
    s["lam"].fill_(lam)
    s["r"] = (2 + 0.25 * s["r"].float()).to(dtype)
    tol = fast_tolerance(lam)
    y, hf, g = both(s)
    ref, grads = reference(s["x"], s["r"], s["i"], s["lam"], s["reset"], s["h0"], s["dy"], s["dhf"])
    assert off_by_channel(y, ref) <= tol and off_by_channel(hf, ref[:, -1], ref) <= tol
    for k in ("dx", "dr", "di", "dh0"):
        assert off_by_channel(g[k], grads[k]) <= tol, k
    gap = np.abs(g["dlam"].double().cpu().numpy() - np.asarray(grads["dlam"]))
    assert np.all(gap <= tol * grads["dlam"].magnitude)


@pytest.mark.parametrize("lam", [-3.0, 0.0, 2.0, 4.0])
def test_a_decay_by_itself(lam):
    """Without input a state is multiplied by its decays, down to e^-96: by the
    scan and by the step."""
    import selective_state_space_12_b200 as ssd

    s = make(2, 3, 130, seed=10)
    s["lam"].fill_(lam)
    s["x"].zero_()
    ref, _ = reference(s["x"], s["r"], s["i"], s["lam"], None, s["h0"])
    y, _, _ = both(s)
    h = s["h0"].clone()
    for t in range(3):
        x, r, i = (s[k][:, t].contiguous() for k in ("x", "r", "i"))
        y1 = ssd.ssd_gated_step(h, x, r, i, s["lam"])
        tol = (t + 1) * fast_tolerance(lam)
        for got in (y[:, t], y1, h):
            gap = np.abs(got.double().cpu().numpy() - ref[:, t])
            assert np.all(gap <= tol * np.abs(ref[:, t]) + 2.0 ** -126)  # below: not held
