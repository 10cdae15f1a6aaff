"""Calls with stream= on two streams, from a third, with nothing waited for in
between: they run at the same time, and what each gives equals what it gives
alone, to the bit.

But for dB and dC of the layer's backward pass: the tensor-core kernels add the
heads' terms to them in memory, in an order that changes. Two orders of a sum of
n terms differ by at most 2 (n - 1) half steps (2^-24) of the terms' magnitudes,
which calls for one head at a time give."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_12_b200 import build

    build.build()


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def gated(seed, L=6000, D=333):
    import selective_state_space_12_b200 as ssd

    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, i, dy = (normal(g, 1, L, D) for _ in range(4))
    lam = -4.5 + 0.1 * normal(g, D, dtype=torch.float32)
    saved, states = ssd.GatedCheckpoint8(1, L, D), torch.empty((1, ssd.gated_blocks(L), D), device="cuda")
    ssd.ssd_gated_scan(x, r, i, lam, checkpoint=saved)
    ssd.ssd_gated_scan(x, r, i, lam, states=states)
    h = normal(g, 300, D, dtype=torch.float32)
    return dict(
        gated_scan=lambda **k: ssd.ssd_gated_scan(x, r, i, lam, **k),
        gated_scan_backward=lambda **k: ssd.ssd_gated_scan_backward(x, r, i, lam, states, dy, **k),
        gated_scan_backward_ckpt8=lambda **k: ssd.ssd_gated_scan_backward_ckpt8(saved, lam, dy, **k),
        gated_step=lambda **k: ssd.ssd_gated_step(h.clone(), x[0, :300].contiguous(),
                                                  r[0, :300].contiguous(), i[0, :300].contiguous(),
                                                  lam, **k))


def selective(seed, L=700, D=512, N=16):
    import selective_state_space_12_b200 as ssd

    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dt, dy = (normal(g, 2, L, D) for _ in range(3))
    A = -torch.exp(normal(g, D, N, dtype=torch.float32))
    B, C = (normal(g, 2, L, 1, N) for _ in range(2))
    bias = torch.full((D,), -4.0, device="cuda")
    return dict(
        selective_scan=lambda **k: ssd.ssd_selective_scan(x, dt, A, B, C, dt_bias=bias,
                                                          dt_softplus=True, **k),
        selective_scan_backward=lambda **k: ssd.ssd_selective_scan_backward(
            x, dt, A, B, C, None, None, dy, dt_bias=bias, dt_softplus=True, zoh=True, **k))


def heads_apart(s, dy, k):
    """The sum over heads of the magnitudes of their terms of dB or dC."""
    import selective_state_space_12_b200 as ssd

    x, dt, A, B, C = s
    cut = lambda t, h: t[:, :, h:h + 1].contiguous()
    return sum(ssd.ssd_backward(cut(x, h), cut(dt, h), A[h:h + 1].contiguous(), B, C, None, None,
                                cut(dy, h))[k].abs() for h in range(len(A)))


def layer(seed, b=2, L=600, H=8, P=64, N=128):
    import selective_state_space_12_b200 as ssd

    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = normal(g, b, L, H, P), normal(g, b, L, H, P)
    dt = torch.rand((b, L, H), generator=g, device="cuda").mul(0.1).bfloat16()
    A = -torch.exp(normal(g, H, dtype=torch.float32))
    B, C = normal(g, b, L, 1, N), normal(g, b, L, 1, N)
    h = normal(g, b, H, P, N, dtype=torch.float32)
    s = (x, dt, A, B, C)
    return dict(
        slack=lambda: {k: 2 * (H - 1) * 2.0 ** -24 * heads_apart(s, dy, k) for k in ("dB", "dC")},
        forward=lambda **k: ssd.ssd_forward(x, dt, A, B, C, **k),
        forward_ex=lambda **k: ssd.ssd_forward_ex(x, dt, A, B, C, zoh=True, **k),
        forward_state=lambda **k: ssd.ssd_forward_state(x, dt, A, B, **k),
        backward=lambda **k: ssd.ssd_backward(x, dt, A, B, C, None, None, dy, **k),
        step=lambda **k: ssd.ssd_step(h.clone(), x[:, 0].contiguous(), dt[:, 0].contiguous(), A,
                                      B[:, 0].contiguous(), C[:, 0].contiguous(), **k))


MAKERS = {**{"gated_" + k: (gated, "gated_" + k) for k in ("scan", "scan_backward",
                                                           "scan_backward_ckpt8", "step")},
          **{k: (selective, k) for k in ("selective_scan", "selective_scan_backward")},
          **{k: (layer, k) for k in ("forward", "forward_ex", "forward_state", "backward", "step")}}


@pytest.mark.parametrize("name", sorted(MAKERS))
def test_two_streams_at_once(name):
    import selective_state_space_12_b200 as ssd

    make, key = MAKERS[name]
    made = [make(1), make(2)]
    calls = [m[key] for m in made]
    want = [[t.clone() for t in tensors(c())] for c in calls]
    slack = [[None] * len(w) for w in want]
    if name == "backward":  # dx, ddt, dA, dB, dC, dD, dh0
        for m, room in zip(made, slack):
            room[3], room[4] = m["slack"]().values()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(4):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)  # about 1 ms: both calls are in line before either runs
        got.append([tensors(c(stream=s)) for c, s in zip(calls, streams)])
        spoil = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(8)]
        del spoil
    torch.cuda.synchronize()
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
    for run in got:
        for w, g, room in zip(want, run, slack):
            assert len(w) == len(g)
            for k, (a, b, r) in enumerate(zip(w, g, room)):
                same = torch.equal(a, b) if r is None else bool(((a - b).abs() <= r).all())
                assert same, (k, float((a - b).abs().max()))


def test_inputs_dropped_after_the_call():
    """Inputs made for the call only, dropped while it is still in line."""
    import selective_state_space_12_b200 as ssd

    s = torch.cuda.Stream()
    x = torch.randn((1, 3000, 256), device="cuda").bfloat16()
    lam = torch.full((256,), -4.5, device="cuda")
    want, _ = ssd.ssd_gated_scan(x, x, x, lam)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(4_000_000)
    s.wait_stream(torch.cuda.current_stream())
    copies = [x.clone() for _ in range(3)]
    s.wait_stream(torch.cuda.current_stream())
    y, _ = ssd.ssd_gated_scan(*copies, lam, stream=s)
    del copies
    others = [torch.zeros_like(x) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(others) == 4


def test_a_side_stream_inside_a_capture():
    """Calls on a stream that a capture has forked to, twice with an empty cache in
    between, replayed beside eager calls."""
    import selective_state_space_12_b200 as ssd

    calls = [gated(3)["gated_scan"], gated(4)["gated_scan_backward"],
             selective(5)["selective_scan_backward"], layer(6)["forward"]]
    want = [[t.clone() for t in tensors(c())] for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph, side = torch.cuda.CUDAGraph(), [torch.cuda.Stream() for _ in calls]
        with torch.cuda.graph(graph):
            now = torch.cuda.current_stream()
            got = []
            for c, s in zip(calls, side):
                s.wait_stream(now)
                got.append(tensors(c(stream=s)))
            for s in side:
                now.wait_stream(s)
        graphs.append((graph, got))
        torch.cuda.empty_cache()
    for _ in range(2):
        for graph, got in graphs:
            for t in (t for out in got for t in out):
                t.zero_()
            graph.replay()
            eager = tensors(calls[0]())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
            for w, g in zip(want, got):
                assert all(torch.equal(a, b) for a, b in zip(w, g))
    assert ssd.ssd_device_status() == 0, ssd.ssd_last_error()
