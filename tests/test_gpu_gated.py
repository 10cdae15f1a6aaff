"""The gated recurrence on the GPU against its definition in 64 bits, token
after token: forward, backward, one-token step and 8-bit checkpoints.

An output's error is what is left of |got - ref| after its own rounding, half a
step of its type relative to its value (bf16 2^-8, fp32 2^-24), as a share of
the larger of the value and the rms. It is held to 2e-5: the gates are within
about 2^-21 (5e-7) of their values, which a state that remembers M tokens sees
through sums, not products, of relative errors, and the states' own roundings,
2^-24 a token, add up over at most about 1000 remembered tokens with random
signs (32 x 6e-8 = 2e-6); a factor of ten is left for the largest of many.
(A share of the rms alone would not hold: a bf16 value of 14 rms is rounded by
up to 14 x 2^-8 = 0.055 rms, and a token after a reset, where m = 1, has such
gradients.)"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

C = 8.0
BLOCK = 64
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_12_b200 import build

    build.build()


def make(b, L, D, dtype=F32, reset=False, h0=True, seed=0, strong=False):
    """Inputs on the GPU; ``strong``: decays down to about e^-20 a token."""
    g = np.random.default_rng(seed)

    def t(a, dt=F32):
        return torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda().to(dt)

    keep = -np.log(g.uniform(0.9, 0.999, D)) / C
    if strong:
        keep = np.exp(g.uniform(np.log(1e-3), np.log(2.5), D))
    s = dict(x=t(g.standard_normal((b, L, D)), dtype), r=t(2 * g.standard_normal((b, L, D)), dtype),
             i=t(2 * g.standard_normal((b, L, D)), dtype), lam=t(np.log(np.expm1(keep))),
             dy=t(g.standard_normal((b, L, D)), dtype), h0=None, dhf=None, reset=None)
    if h0:
        s["h0"], s["dhf"] = t(g.standard_normal((b, D))), t(g.standard_normal((b, D)))
    if reset:
        s["reset"] = torch.from_numpy((g.random((b, L)) < 0.02).astype(np.uint8)).cuda()
    return s


class Sum(np.ndarray):
    """A sum over batch and tokens that knows the sum of its terms' magnitudes."""

    def __new__(cls, terms):
        v = terms.sum((0, 1)).view(cls)
        v.magnitude = np.abs(terms).sum((0, 1))
        return v


def reference(x, r, i, lam, reset, h0, dy=None, dhf=None, states=None, c=C):
    """(h, gradients) in 64 bits; with states, each block of 64 tokens starts from its own."""
    f = lambda v: None if v is None else v.detach().double().cpu().numpy()
    x, r, i, lam, h0, dy, dhf, states = map(f, (x, r, i, lam, h0, dy, dhf, states))
    b, L, D = x.shape
    sr, si = 1 / (1 + np.exp(-r)), 1 / (1 + np.exp(-i))
    sp = np.logaddexp(lam, 0)
    s = -c * sp * sr
    a, m = np.exp(s), np.sqrt(-np.expm1(2 * s))
    rs = np.zeros((b, L), bool) if reset is None else reset.cpu().numpy() != 0
    a, m = np.where(rs[..., None], 0, a), np.where(rs[..., None], 1, m)
    h, before = np.zeros((b, L, D)), np.zeros((b, L, D))
    cur = np.zeros((b, D)) if h0 is None else h0
    for t in range(L):
        if states is not None and t % BLOCK == 0:
            cur = states[:, t // BLOCK]
        before[:, t] = cur
        cur = np.where(rs[:, t, None], 0, a[:, t] * cur) + m[:, t] * si[:, t] * x[:, t]
        h[:, t] = cur
    if dy is None:
        return h, None
    G = np.zeros((b, L, D))
    carry = np.zeros((b, D)) if dhf is None else dhf
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + carry
        carry = np.where(rs[:, t, None], 0, a[:, t] * G[:, t])
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(m > 0, a * a / m, 0)
    ds = np.where(rs[..., None], 0, G * (a * before - ratio * si * x))
    terms = -ds * c * sr / (1 + np.exp(-lam))
    return h, dict(dx=G * m * si, dr=ds * s * (1 - sr), di=G * m * x * si * (1 - si),
                   dlam=Sum(terms), dh0=carry)


TOL = 2e-5


def off(got, ref):
    half = torch.finfo(got.dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape
    if not ref.size:
        return 0.0
    size = np.maximum(np.abs(ref), max(np.sqrt(np.mean(np.square(ref))), 1e-300))
    if isinstance(ref, Sum):
        # terms of both signs cancel: each is a product of four factors (a gate, s a, G and h)
        # within about 5e-7 of their values, so the sum is within 2e-6 of the terms' magnitudes
        size, ref = np.maximum(np.asarray(size), ref.magnitude * (2e-6 / TOL)), np.asarray(ref)
    return float(np.max(np.maximum(np.abs(got - ref) - half * np.abs(ref), 0) / size))


def forward(s, **kw):
    import selective_state_space_12_b200 as ssd

    b, L, D = s["x"].shape
    states = torch.full((b, ssd.gated_blocks(L), D), float("nan"), device="cuda")
    y, hf = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                               states=states, **kw)
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    return y, hf, states


SHAPES = [(1, 1, 1), (1, 1, 64), (2, 2, 3), (1, 63, 65), (3, 64, 128), (1, 65, 130), (2, 129, 62),
          (1, 200, 1001), (2, 1000, 257), (4, 515, 66), (1, 4100, 40), (2, 3000, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, reset, dtype):
    s = make(*shape, dtype=dtype, reset=reset, seed=sum(shape))
    h, _ = reference(s["x"], s["r"], s["i"], s["lam"], s["reset"], s["h0"])
    y, hf, states = forward(s)
    assert off(y, h) <= TOL
    assert off(hf, h[:, -1]) <= TOL
    entering = np.concatenate([s["h0"].double().cpu().numpy()[:, None],
                               h[:, BLOCK - 1:-1:BLOCK]], 1)
    assert off(states, entering) <= TOL


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, reset, dtype):
    import selective_state_space_12_b200 as ssd

    s = make(*shape, dtype=dtype, reset=reset, h0=shape[0] != 3, seed=10 + sum(shape))
    _, _, states = forward(s)
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], states, s["dy"], s["dhf"],
                                    reset=s["reset"])
    assert ssd.ssd_device_status() == 0
    _, ref = reference(s["x"], s["r"], s["i"], s["lam"], s["reset"], s["h0"], s["dy"], s["dhf"])
    for k, v in ref.items():
        if np.any(v):
            assert off(g[k], v) <= TOL, k
        else:
            assert not g[k].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strong_decays(dtype):
    import selective_state_space_12_b200 as ssd

    s = make(2, 300, 96, dtype=dtype, seed=77, strong=True)
    h, ref = reference(s["x"], s["r"], s["i"], s["lam"], None, s["h0"], s["dy"], s["dhf"])
    y, hf, states = forward(s)
    assert off(y, h) <= TOL and off(hf, h[:, -1]) <= TOL
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], states, s["dy"], s["dhf"])
    for k, v in ref.items():
        assert off(g[k], v) <= TOL, k


def test_gradients_against_differences():
    """Central differences of the 64-bit definition in random directions; the
    step 1e-4 leaves 1e-8 of truncation, the fp32 gradients 2e-5."""
    import selective_state_space_12_b200 as ssd

    s = make(2, 130, 24, reset=True, seed=5)
    _, _, states = forward(s)
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], states, s["dy"], s["dhf"],
                                    reset=s["reset"])
    rng = np.random.default_rng(6)
    dy, dhf = s["dy"].double().cpu().numpy(), s["dhf"].double().cpu().numpy()

    def loss(**change):
        v = {k: (change[k] if k in change else s[k].double().cpu()) for k in
             ("x", "r", "i", "lam", "h0")}
        h, _ = reference(v["x"], v["r"], v["i"], v["lam"], s["reset"], v["h0"])
        return float((dy * h).sum() + (dhf * h[:, -1]).sum())

    for k, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("h0", "dh0")):
        base = s[k].double().cpu()
        v = torch.from_numpy(rng.standard_normal(tuple(base.shape)))
        eps = 1e-4
        num = (loss(**{k: base + eps * v}) - loss(**{k: base - eps * v})) / (2 * eps)
        got = g[grad].double().cpu()
        scale = float(got.norm() * v.norm())
        assert abs(float((got * v).sum()) - num) <= 1e-4 * scale, k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 2), (2, 64, 70), (1, 200, 33), (3, 130, 256)])
def test_checkpoint_holds_the_inputs_in_8_bits(shape, dtype):
    import selective_state_space_12_b200 as ssd

    s = make(*shape, dtype=dtype, seed=21)
    s["x"][:, :, 0] = 0.0
    s["r"][0, :, 1] *= 1e-3
    s["i"][:, 0, 0] = 127.0 / 64  # the largest that the step below still holds
    ck = ssd.GatedCheckpoint8(*shape)
    y, hf = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], h0=s["h0"], checkpoint=ck)
    assert ssd.ssd_device_status() == 0
    for got, v in zip(ck.values(), (s["x"], s["r"], s["i"])):
        v = v.double().cpu().numpy()
        want = np.zeros_like(v)
        for t in range(0, shape[1], BLOCK):
            part = v[:, t:t + BLOCK]
            top = np.abs(part).max(1, keepdims=True)
            e = np.ceil(np.log2(np.maximum(top, 1e-30) / 127))
            e = np.where(127 * 2.0 ** e < top, e + 1, e)
            e = np.where(127 * 2.0 ** (e - 1) >= top, e - 1, e)
            want[:, t:t + BLOCK] = np.round(part / 2 ** e) * 2 ** e
        assert np.array_equal(got.double().cpu().numpy(), want)
    y2, hf2, states = forward(s)
    assert torch.equal(y, y2) and torch.equal(hf, hf2) and torch.equal(ck.states, states)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 2), (2, 64, 70), (1, 200, 33), (3, 130, 256),
                                   (2, 1000, 100)])
def test_backward_from_the_checkpoint(shape, reset, dtype):
    import selective_state_space_12_b200 as ssd

    s = make(*shape, dtype=dtype, reset=reset, seed=31)
    ck = ssd.GatedCheckpoint8(*shape)
    ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                       checkpoint=ck)
    g = ssd.ssd_gated_scan_backward_ckpt8(ck, s["lam"], s["dy"], s["dhf"], reset=s["reset"])
    assert ssd.ssd_device_status() == 0
    _, ref = reference(*ck.values(), s["lam"], s["reset"], None, s["dy"], s["dhf"], ck.states)
    for k, v in ref.items():
        assert off(g[k], v) <= TOL, k


def test_checkpoint_of_infinities_reads_as_nan():
    import selective_state_space_12_b200 as ssd

    s = make(1, 130, 8, seed=41)
    s["x"][0, 3, 2], s["x"][0, 70, 5] = float("inf"), float("nan")
    ck = ssd.GatedCheckpoint8(1, 130, 8)
    ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], h0=s["h0"], checkpoint=ck)
    bad = torch.isnan(ck.values()[0])
    want = torch.zeros_like(bad)
    want[0, :64, 2] = want[0, 64:128, 5] = True
    assert torch.equal(bad, want) and not any(torch.isnan(v).any() for v in ck.values()[1:])
    g = ssd.ssd_gated_scan_backward_ckpt8(ck, s["lam"], s["dy"], s["dhf"])
    assert torch.isnan(g["dlam"][[2, 5]]).all() and torch.isfinite(g["dlam"][[0, 1, 3, 4, 6, 7]]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 2560), (3, 1001), (256, 130), (301, 2602),
                                   (301, 2601)])
def test_step(shape, dtype):
    import selective_state_space_12_b200 as ssd

    b, D = shape
    s = make(b, 5, D, dtype=dtype, seed=51)
    ref, _ = reference(s["x"], s["r"], s["i"], s["lam"], None, s["h0"])
    h = s["h0"].clone()
    for t in range(5):
        x, r, i = (s[k][:, t].contiguous() for k in ("x", "r", "i"))
        y = ssd.ssd_gated_step(h, x, r, i, s["lam"])
        assert off(y, ref[:, t]) <= TOL and off(h, ref[:, t]) <= TOL


def test_extreme_gates():
    """Shut and open gates, a decay of one and of zero: finite throughout, and
    the limits' values."""
    import selective_state_space_12_b200 as ssd

    L, D = 70, 6
    x = torch.ones((1, L, D), device="cuda")
    r = torch.zeros((1, L, D), device="cuda")
    i = torch.zeros((1, L, D), device="cuda")
    lam = torch.tensor([-200.0, 100.0, 0.0, 0.0, 0.0, 0.0], device="cuda")
    r[..., 2], r[..., 3] = -1e30, 1e30
    i[..., 4], i[..., 5] = -1e30, float("inf")
    h0 = torch.full((1, D), 2.0, device="cuda")
    states = torch.empty((1, 2, D), device="cuda")
    y, hf = ssd.ssd_gated_scan(x, r, i, lam, h0=h0, states=states)
    g = ssd.ssd_gated_scan_backward(x, r, i, lam, states, x, h0)
    assert all(torch.isfinite(v).all() for v in (y, hf, *g.values()))
    assert (y[..., 0] == 2).all()                              # softplus(-200) = 0: a = 1, m = 0
    assert torch.allclose(y[0, 1:, 1], torch.full((L - 1,), 0.5, device="cuda"))  # a = 0
    assert torch.allclose(y[..., 2], torch.full_like(y[..., 2], 2.0), atol=1e-6)
    assert (y[0, 10:, 4].abs() < 1e-6).all()


def test_nothing_passes_a_reset():
    """Infinities and NaN before a reset, and NaN gradients after it, stay
    there; a reset at the first token hides the initial state."""
    import selective_state_space_12_b200 as ssd

    b, L, D = 3, 300, 10
    s = make(b, L, D, seed=61)
    reset = torch.zeros((b, L), dtype=torch.uint8, device="cuda")
    reset[:, 0] = reset[0, 100] = reset[0, 128] = reset[1, 255] = reset[2, 100] = reset[:, -1] = 7
    s["reset"], s["h0"] = reset, torch.full((b, D), float("nan"), device="cuda")
    clean, _, _ = forward(s)
    assert torch.isfinite(clean).all()
    s["x"][0, 40], s["r"][0, 90], s["x"][1, 200] = float("inf"), float("nan"), float("nan")
    s["r"][2, 90] = float("nan")  # a decay that is NaN, in the block and run of a reset
    y, hf, states = forward(s)
    for row, start in ((0, 100), (1, 255), (2, 100)):
        assert torch.equal(y[row, start:], clean[row, start:])
    assert torch.equal(y[0, :40], clean[0, :40]) and torch.isnan(y[1, 210]).all()
    assert torch.isfinite(hf).all()
    s = make(b, L, D, seed=61)
    s["reset"] = reset
    _, _, states = forward(s)
    args = (s["x"], s["r"], s["i"], s["lam"], states)
    ok = ssd.ssd_gated_scan_backward(*args, s["dy"], s["dhf"], reset=reset)
    s["dy"][0, 150] = s["dy"][2, 103] = float("nan")
    g = ssd.ssd_gated_scan_backward(*args, s["dy"], s["dhf"], reset=reset)
    for k in ("dx", "dr", "di"):
        assert torch.equal(g[k][0, :128], ok[k][0, :128]) and torch.equal(g[k][1], ok[k][1])
        assert torch.equal(g[k][0, 151:], ok[k][0, 151:])
        assert torch.equal(g[k][2, :100], ok[k][2, :100]) and torch.isnan(g[k][2, 101:104]).all()
    assert not g["dh0"].any()


def test_empty_sequence():
    import selective_state_space_12_b200 as ssd

    e = torch.empty((2, 0, 6), device="cuda")
    lam, h0 = torch.zeros(6, device="cuda"), torch.randn((2, 6), device="cuda")
    y, hf = ssd.ssd_gated_scan(e, e, e, lam, h0=h0)
    assert y.shape == (2, 0, 6) and torch.equal(hf, h0)
    _, hf = ssd.ssd_gated_scan(e, e, e, lam)
    assert not hf.any()
    g = ssd.ssd_gated_scan_backward(e, e, e, lam, torch.empty((2, 0, 6), device="cuda"), e, h0)
    assert torch.equal(g["dh0"], h0) and not g["dlam"].any() and g["dx"].numel() == 0


def test_slices_that_are_aligned_to_their_elements_only():
    import selective_state_space_12_b200 as ssd

    s = make(1, 140, 64, dtype=BF16, reset=True, seed=71)
    want, _, st = forward(s)
    wg = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"],
                                     reset=s["reset"])

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return buf.copy_(t)

    for k in ("x", "r", "i", "dy"):
        s[k] = shifted(s[k])
    y, _, st2 = forward(s, y=shifted(want).zero_())
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st2, s["dy"], s["dhf"],
                                    reset=s["reset"])
    assert torch.equal(y, want)
    for k in wg:
        assert torch.equal(g[k], wg[k]), k


def test_another_stream_and_a_captured_graph():
    """A side stream, and a graph replayed on new inputs beside eager calls,
    with one workspace for both directions of the graph."""
    import selective_state_space_12_b200 as ssd

    s = make(2, 700, 130, dtype=BF16, reset=True, seed=81)
    want, _, st = forward(s)
    wg = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"],
                                     reset=s["reset"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, _ = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                               stream=side)
    side.synchronize()
    assert torch.equal(y2, want)

    bufs = {k: torch.zeros_like(s[k]) for k in ("x", "r", "i", "dy")}
    ck = ssd.GatedCheckpoint8(2, 700, 130)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, hfg = ssd.ssd_gated_scan(bufs["x"], bufs["r"], bufs["i"], s["lam"], reset=s["reset"],
                                     h0=s["h0"], checkpoint=ck)
        gg = ssd.ssd_gated_scan_backward(bufs["x"], bufs["r"], bufs["i"], s["lam"], ck.states,
                                         bufs["dy"], s["dhf"], reset=s["reset"])
    for _ in range(3):
        for k in bufs:
            bufs[k].copy_(s[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, want)
        for k in wg:
            assert torch.equal(gg[k], wg[k]), k
        for t in bufs.values():
            t.zero_()
        graph.replay()
    assert ssd.ssd_device_status() == 0


def test_repeats_to_the_bit_and_h_final_may_be_h0():
    import selective_state_space_12_b200 as ssd

    s = make(3, 2000, 500, dtype=BF16, seed=91)
    y, hf, st = forward(s)
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"])
    for _ in range(4):
        h = s["h0"].clone()
        y2, hf2 = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], h0=h, h_final=h)
        assert torch.equal(y2, y) and torch.equal(h, hf)
        g2 = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"])
        for k in g:
            assert torch.equal(g2[k], g[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("batch,L,D", [(4, 1100, 1024), (5, 1100, 1030), (2, 700, 2600)])
def test_as_many_lanes_as_half_the_sms(batch, L, D, dtype):
    """Lanes (of 64 channels) just below and above half the SMs, fewer than thread
    blocks: the chain of waits is as long as the sequence."""
    import selective_state_space_12_b200 as ssd

    s = make(batch, L, D, dtype=dtype, reset=True, seed=93)
    y, hf, st = forward(s)
    g = ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], st, s["dy"], s["dhf"],
                                    reset=s["reset"])
    saved = ssd.GatedCheckpoint8(batch, L, D)
    y8, _ = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], reset=s["reset"], h0=s["h0"],
                               checkpoint=saved)
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    assert torch.equal(y8, y)
    ref, grads = reference(s["x"], s["r"], s["i"], s["lam"], s["reset"], s["h0"], s["dy"], s["dhf"])
    assert off(y, ref) <= TOL and off(hf, ref[:, -1]) <= TOL
    for k in grads:
        assert off(g[k], grads[k]) <= TOL, k


@pytest.mark.parametrize("batch,L,D", [(1, 40, 70), (1, 65, 128), (2, 500, 64), (1, 513, 200),
                                       (1, 4000, 64), (40, 130, 1024)])
def test_the_end_may_take_the_starts_place(batch, L, D):
    """h_final in h0's memory and dh0 in dh_final's, with one block of tokens, one
    group of blocks, several, and more lanes than thread blocks."""
    import selective_state_space_12_b200 as ssd
    from selective_state_space_12_b200 import _lib
    from selective_state_space_12_b200.ssd import make_dims

    s = make(batch, L, D, dtype=BF16, seed=92)
    args = (s["x"], s["r"], s["i"], s["lam"])
    y, hf, st = forward(s)
    g = ssd.ssd_gated_scan_backward(*args, st, s["dy"], s["dhf"])
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    at = lambda t: t.data_ptr()
    dims = ctypes.byref(make_dims(batch, L, D, 1, 1, 1, BF16))
    need = lib.ssd_gated_scan_backward_workspace_size(dims)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        h = s["h0"].clone()
        y2, _ = ssd.ssd_gated_scan(*args, h0=h, h_final=h)
        assert torch.equal(y2, y) and torch.equal(h, hf)
        d = s["dhf"].clone()
        out = {k: torch.empty_like(g[k]) for k in ("dx", "dr", "di", "dlam")}
        assert lib.ssd_gated_scan_backward(
            *(at(t) for t in args[:3]), None, None, at(s["lam"]), C, None, at(st), at(s["dy"]),
            at(d), at(out["dx"]), at(out["dr"]), at(out["di"]), at(out["dlam"]), at(d), dims,
            at(ws), need, stream) == 0
        assert torch.equal(d, g["dh0"])
        for k in out:
            assert torch.equal(out[k], g[k]), k


def test_prefill_then_steps_and_a_split_sequence():
    """As used for generation: a prompt in two calls, then single tokens, gives
    the whole sequence's outputs."""
    import selective_state_space_12_b200 as ssd

    s = make(2, 300, 192, dtype=BF16, seed=101)
    whole, hf, _ = forward(s)
    cut = lambda a, b: [s[k][:, a:b].contiguous() for k in ("x", "r", "i")]
    y1, h = ssd.ssd_gated_scan(*cut(0, 137), s["lam"], h0=s["h0"])
    y2, h = ssd.ssd_gated_scan(*cut(137, 290), s["lam"], h0=h)
    ys = [y1, y2]
    for t in range(290, 300):
        x, r, i = (s[k][:, t].contiguous() for k in ("x", "r", "i"))
        ys.append(ssd.ssd_gated_step(h, x, r, i, s["lam"])[:, None])
    y = torch.cat(ys, 1)
    ref, _ = reference(s["x"], s["r"], s["i"], s["lam"], None, s["h0"])
    assert off(y, ref) <= TOL and off(whole, ref) <= TOL
    assert off(h, ref[:, -1]) <= TOL and off(hf, ref[:, -1]) <= TOL


def test_a_large_problem_past_32_bit_offsets():
    """b L D = 2.2e9: the last rows lie beyond 2^31 elements; checked on
    sampled channels."""
    import selective_state_space_12_b200 as ssd

    b, L, D = 2, 131072, 8448
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((b, L, D), generator=g, device="cuda", dtype=BF16)
    lam = torch.full((D,), -4.5, device="cuda")
    y, hf = ssd.ssd_gated_scan(x, x, x, lam)
    assert ssd.ssd_device_status() == 0
    for d in (0, 4000, D - 1):
        v = x[1:, :, d:d + 1]
        ref, _ = reference(v, v, v, lam[d:d + 1], None, None)
        assert off(y[1:, :, d:d + 1], ref) <= TOL
        end = abs(float(hf[1, d]) - ref[0, -1, 0])
        assert end <= TOL * np.sqrt(np.mean(ref * ref))


@pytest.mark.parametrize("batch,L,D", [(2, 4000, 2600), (2, 4000, 2601)])
def test_waits_run_out_with_many_lanes_then_recover(batch, L, D):
    """The same with a lane for every other SM, rows ahead on their way."""
    import selective_state_space_12_b200 as ssd

    s = make(batch, L, D, dtype=BF16, seed=112)
    want, _, st = forward(s)
    args = (s["x"], s["r"], s["i"], s["lam"])
    g = ssd.ssd_gated_scan_backward(*args, st, s["dy"])
    saved = ssd.GatedCheckpoint8(batch, L, D)
    ssd.ssd_gated_scan(*args, checkpoint=saved)
    for call in (lambda: ssd.ssd_gated_scan(*args, h0=s["h0"]),
                 lambda: ssd.ssd_gated_scan_backward(*args, st, s["dy"]),
                 lambda: ssd.ssd_gated_scan_backward_ckpt8(saved, s["lam"], s["dy"])):
        ssd.ssd_set_wait_limit(16)
        try:
            call()
            status, msg = ssd.ssd_device_status(), ssd.ssd_last_error()
        finally:
            ssd.ssd_set_wait_limit(0)
        assert status == 5 and "gave up" in msg
        assert ssd.ssd_device_status() == 0
    y, _, _ = forward(s)
    assert torch.equal(y, want)
    again = ssd.ssd_gated_scan_backward(*args, st, s["dy"])
    for k in g:
        assert torch.equal(g[k], again[k]), k


def test_look_back_wait_runs_out_then_recovers():
    """Few channels and a long sequence: thread blocks wait for the ones before
    them. With a bound of a few cycles the call reports a time-out; the next one
    computes as before."""
    import selective_state_space_12_b200 as ssd

    s = make(1, 20000, 64, dtype=BF16, seed=111)
    want, _, st = forward(s)
    args = (s["x"], s["r"], s["i"], s["lam"])
    for call in (lambda: ssd.ssd_gated_scan(*args, h0=s["h0"]),
                 lambda: ssd.ssd_gated_scan_backward(*args, st, s["dy"])):
        ssd.ssd_set_wait_limit(16)
        try:
            call()
            status, msg = ssd.ssd_device_status(), ssd.ssd_last_error()
        finally:
            ssd.ssd_set_wait_limit(0)
        assert status == 5 and "gave up" in msg
        assert ssd.ssd_device_status() == 0
    y, _, _ = forward(s)
    assert torch.equal(y, want)


def test_calls_at_once_on_several_streams():
    """Calls of both ways of chaining overlap on three streams, thread blocks of
    one waiting while the others' run: the same results to the bit."""
    import selective_state_space_12_b200 as ssd

    cases = [make(1, 9000, 512, dtype=BF16, seed=121), make(2, 1500, 2600, dtype=BF16, seed=122),
             make(1, 7000, 333, reset=True, seed=123)]

    def call(s):
        st = torch.empty((s["x"].shape[0], ssd.gated_blocks(s["x"].shape[1]), s["x"].shape[2]),
                         device="cuda")
        args = (s["x"], s["r"], s["i"], s["lam"])
        y, hf = ssd.ssd_gated_scan(*args, reset=s["reset"], h0=s["h0"], states=st)
        g = ssd.ssd_gated_scan_backward(*args, st, s["dy"], s["dhf"], reset=s["reset"])
        return [y, hf, st] + [g[k] for k in ("dx", "dr", "di", "dlam", "dh0")]

    want = [call(s) for s in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for k, (s, stream) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(stream):
                got[k].append(call(s))
    torch.cuda.synchronize()
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    for w, runs in zip(want, got):
        for run in runs:
            for a, b in zip(w, run):
                assert torch.equal(a, b)
