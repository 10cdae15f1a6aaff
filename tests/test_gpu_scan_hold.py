"""The zero-order hold's gradients of A and of the steps over the whole range of
z = dt A, where their terms cancel: against the 64-bit adjoint of the selective
scan's other tests, held to their bound, 2e-4.

What the kernel's forms lose, of a term's size: near 0 the form of w - dt leaves
out z^3/360 of it, 1.7e-5 where the other takes over, which loses 2^-22 / (z^2/2)
there, 1.4e-5; at z = -96 that loses 96 x 2^-24 a rounding, 2.3e-5 for four; and
with a = exp(z) above e^-4 a sum of a's size keeps 2^-24 / a, 3e-6 a rounding."""
import numpy as np
import pytest

from test_gpu_scan_backward import BF16, F32, TOL, f64, make, off, reference, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_12_b200 import build

    build.build()


def put(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda()


def by_channel(got, ref):
    """The error as a share of the larger of the value and its channel's rms."""
    got = f64(got)
    size = np.maximum(np.abs(ref), np.sqrt(np.mean(ref * ref, axis=(0, 1))))
    return float(np.max(np.abs(got - ref) / np.maximum(size, 1e-300)))


def holds(s, **o):
    g, ref = run(s, zoh=True, **o), reference(s, zoh=True, **o)
    # what lies below fp32's least normal number (dh0 after a hundred fast decays) is not held
    ref = {k: np.where(np.abs(v) < 2.0 ** -126, 0, v) for k, v in ref.items()}
    far = {k: off(g[k], v) for k, v in ref.items() if np.any(v)}
    far["ddt of each channel"] = by_channel(g["ddt"], ref["ddt"])
    assert all(v <= TOL for v in far.values()), {k: v for k, v in far.items() if v > TOL}


@pytest.mark.parametrize("L", [1, 8, 64, 200])
@pytest.mark.parametrize("step", [1e-5, 1e-4, 1e-3])
@pytest.mark.parametrize("D,N", [(40, 16), (33, 4), (70, 8)])
def test_small_steps_from_a_zero_state(D, N, step, L):
    """|A| from 2^-5 to 1: the sequence remembers all of its few tokens, and
    dA is second order in the step."""
    g = np.random.default_rng(L + D)
    s = make(2, L, D, N, softplus=False, h0=False, seed=L + N)
    s["A"] = put(-np.exp(g.uniform(np.log(2.0 ** -5), 0, (D, N))))
    s["dt"] = put(step * np.exp(g.uniform(-0.5, 0.5, (2, L, D))))
    holds(s)


def test_small_steps_after_a_masked_stretch():
    """A left-padded batch: zero inputs for long, then a few tokens."""
    s = make(2, 300, 48, 16, softplus=True, h0=False, seed=3)
    s["bias"].fill_(-7.0)
    s["x"][:, :290] = 0.0
    holds(s, softplus=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,N,G", [(40, 16, 1), (96, 16, 3), (66, 4, 2), (32, 8, 1)])
@pytest.mark.parametrize("step", [2.0, 6.0])
def test_every_state_forgets_fast(step, D, N, G, dtype):
    """z from -8 to -50 for all states of a channel: the step's gradient is in
    proportion to exp(z)."""
    g = np.random.default_rng(D)
    s = make(2, 100, D, N, G, dtype=dtype, softplus=False, seed=D + N)
    s["A"] = put(-np.exp(g.uniform(np.log(4), np.log(8), (D, N))))
    s["dt"] = put(step * np.exp(g.uniform(-0.02, 0.02, (2, 100, D)))).to(dtype)
    holds(s)


def test_steps_and_decays_of_all_sizes_at_once():
    g = np.random.default_rng(8)
    s = make(2, 150, 77, 16, softplus=False, seed=9)
    s["A"] = put(-np.exp(g.uniform(np.log(1e-6), np.log(1e4), (77, 16))))
    s["A"][:, 3], s["A"][:, 5], s["A"][:, 7] = 0.0, 0.05, 2.0 ** -45
    s["dt"] = put(np.exp(g.uniform(np.log(1e-4), np.log(2), (2, 150, 77))))
    g_, ref = run(s, zoh=True), reference(s, zoh=True)
    far = {k: off(g_[k], v) for k, v in ref.items() if np.any(v)}
    assert all(v <= TOL for v in far.values()), {k: v for k, v in far.items() if v > TOL}


@pytest.mark.parametrize("A", [-1.0, -16.0, -2.0 ** -6, 1.0])
@pytest.mark.parametrize("N", [4, 16])
def test_one_token_at_every_step(N, A):
    """One token, no state before it, B = C: dA and ddt are one positive term for
    each state, so each entry is held to its own size. dA = r x B dt^2 (z e^z -
    (e^z - 1)) / z^2 and ddt = r x B e^z."""
    D = 512
    z = np.sign(A) * np.exp(np.linspace(np.log(1e-7), np.log(60.0 if A > 0 else 200.0), D))
    hold = z > -80  # exp(z) is a normal number, for ddt
    s = make(1, 1, D, N, softplus=False, h0=False, seed=4, Dskip=False)
    s["A"].fill_(A)
    s["dt"] = put(z / A)[None, None]
    s["C"] = s["B"].clone()
    s["x"], s["dy"] = s["x"].abs() + 0.1, s["dy"].abs() + 0.1
    g, ref = run(s, zoh=True), reference(s, zoh=True)
    for k in ("dA", "ddt", "dx", "dB", "dC"):
        rel = np.abs(f64(g[k]) - ref[k]) / np.abs(ref[k])
        rel = rel[..., hold] if k == "ddt" else rel
        assert rel.max() <= TOL, (k, rel.max())
