"""What the gated scan's entry points refuse, before anything is enqueued (no
GPU needed)."""
import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_12_b200 import build

    build.build()
    from selective_state_space_12_b200 import _lib

    return _lib.load()


def dims(**kw):
    from selective_state_space_12_b200 import _lib

    d = dict(batch=2, seqlen=100, nheads=64, headdim=1, dstate=1, ngroups=1, dtype=1, reserved=0)
    d.update(kw)
    return _lib.Dims(**d)


PTR = {n: 0x10000 * (k + 1) for k, n in enumerate(
    ("x", "r", "i", "lam", "y", "h0", "hf", "states", "q", "e", "dy", "dx", "dr", "di", "dlam",
     "dh0", "h", "ws", "dhf", "reset"))}


def fwd(lib, d=None, c=8.0, ws_bytes=1 << 40, null=(), **kw):
    a = dict(x=PTR["x"], r=PTR["r"], i=PTR["i"], lam=PTR["lam"], reset=None, h0=None, y=PTR["y"],
             hf=None, states=None, q=None, e=None, ws=PTR["ws"])
    a.update(kw)
    return lib.ssd_gated_scan(a["x"], a["r"], a["i"], a["lam"], c, a["reset"], a["h0"], a["y"],
                              a["hf"], a["states"], a["q"], a["e"],
                              ctypes.byref(d or dims()), a["ws"], ws_bytes, None)


def bwd(lib, d=None, c=8.0, ws_bytes=1 << 40, **kw):
    a = {k: PTR[k] for k in ("x", "r", "i", "lam", "states", "dy", "dx", "dr", "di", "dlam", "ws")}
    a.update(q=None, e=None, reset=None, dhf=None, dh0=None)
    a.update(kw)
    return lib.ssd_gated_scan_backward(a["x"], a["r"], a["i"], a["q"], a["e"], a["lam"], c,
                                       a["reset"], a["states"], a["dy"], a["dhf"], a["dx"],
                                       a["dr"], a["di"], a["dlam"], a["dh0"],
                                       ctypes.byref(d or dims()), a["ws"], ws_bytes, None)


def step(lib, d=None, c=8.0, **kw):
    a = {k: PTR[k] for k in ("h", "x", "r", "i", "lam", "y")}
    a.update(kw)
    return lib.ssd_gated_step(a["h"], a["x"], a["r"], a["i"], a["lam"], c, a["y"],
                              ctypes.byref(d or dims()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(nheads=0), INVALID), (dict(seqlen=-1), INVALID),
    (dict(headdim=16), INVALID), (dict(dstate=4), INVALID), (dict(ngroups=2), INVALID),
    (dict(dtype=2), INVALID), (dict(reserved=1), INVALID), (dict(batch=70000), UNSUPPORTED),
    (dict(nheads=(1 << 24) + 1), UNSUPPORTED), (dict(seqlen=(1 << 30) + 1), UNSUPPORTED),
    (dict(batch=60000, nheads=1 << 24, seqlen=1 << 20), UNSUPPORTED),
])
def test_sizes(lib, kw, status):
    assert fwd(lib, dims(**kw)) == status and lib.ssd_last_error()
    assert bwd(lib, dims(**kw)) == status
    if "seqlen" not in kw:
        assert step(lib, dims(**kw)) == status
    assert lib.ssd_gated_scan_workspace_size(ctypes.byref(dims(**kw))) == 0
    assert lib.ssd_gated_scan_backward_workspace_size(ctypes.byref(dims(**kw))) == 0


@pytest.mark.parametrize("c", [0.0, -1.0, float("inf"), float("nan")])
def test_gate_power(lib, c):
    assert fwd(lib, c=c) == bwd(lib, c=c) == step(lib, c=c) == INVALID


def test_missing_and_misaligned_pointers(lib):
    for n in ("x", "r", "i", "lam", "y"):
        assert fwd(lib, **{n: None}) == INVALID
        assert fwd(lib, **{n: 0x10001}) == INVALID
        assert step(lib, **{n: None}) == step(lib, **{n: 0x10001}) == INVALID
    for n in ("h0", "hf", "states"):
        assert fwd(lib, **{n: 0x10002}) == INVALID
    for n in ("x", "r", "i", "lam", "states", "dy", "dx", "dr", "di", "dlam"):
        assert bwd(lib, **{n: None}) == INVALID
        assert bwd(lib, **{n: 0x10001}) == INVALID
    assert step(lib, h=None) == step(lib, h=0x10002) == INVALID


def test_checkpoint_arguments(lib):
    assert fwd(lib, q=PTR["q"]) == fwd(lib, e=PTR["e"]) == INVALID
    assert bwd(lib, q=PTR["q"]) == bwd(lib, e=PTR["e"]) == INVALID
    # both the inputs and their copies
    assert bwd(lib, q=PTR["q"], e=PTR["e"]) == INVALID
    assert b"not both" in lib.ssd_last_error()


def test_aliases(lib):
    for n in ("x", "r", "i"):
        assert fwd(lib, y=PTR[n]) == INVALID and b"aliases" in lib.ssd_last_error()
        assert step(lib, y=PTR[n]) == INVALID
        assert bwd(lib, dx=PTR[n]) == bwd(lib, dr=PTR[n]) == bwd(lib, di=PTR[n]) == INVALID
    assert bwd(lib, dx=PTR["dy"]) == bwd(lib, di=PTR["states"]) == INVALID
    assert fwd(lib, states=PTR["h0"], h0=PTR["h0"]) == INVALID
    assert step(lib, y=PTR["h"]) == INVALID


def test_workspace(lib):
    for call, size in ((fwd, lib.ssd_gated_scan_workspace_size),
                       (bwd, lib.ssd_gated_scan_backward_workspace_size)):
        need = size(ctypes.byref(dims()))
        assert need > 0
        assert call(lib, ws_bytes=need - 1) == INVALID and b"workspace" in lib.ssd_last_error()
        assert call(lib, ws=PTR["ws"] + 16) == INVALID


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import selective_state_space_12_b200 as ssd

    x, lam = torch.zeros((1, 8, 4)), torch.zeros(4)
    st = torch.zeros((1, 1, 4))
    with pytest.raises((ValueError, RuntimeError), match="(?i)cuda"):
        ssd.ssd_gated_scan(x, x, x, lam)
    with pytest.raises((ValueError, RuntimeError), match="(?i)cuda"):
        ssd.ssd_gated_scan_backward(x, x, x, lam, st, x)
    with pytest.raises((ValueError, RuntimeError), match="(?i)cuda"):
        ssd.ssd_gated_step(torch.zeros((1, 4)), x[:, 0].contiguous(), x[:, 0].contiguous(),
                           x[:, 0].contiguous(), lam)
    with pytest.raises(TypeError, match="dtype"):
        ssd.ssd_gated_scan(x, x.bfloat16(), x, lam)
    with pytest.raises(TypeError, match="unsupported I/O dtype"):
        ssd.ssd_gated_scan(x.half(), x.half(), x.half(), lam)
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_gated_scan(x, x[:, :4].contiguous(), x, lam)
    with pytest.raises(ValueError, match="contiguous"):
        ssd.ssd_gated_scan(x, torch.zeros((1, 4, 8)).transpose(1, 2), x, lam)
    with pytest.raises(TypeError, match="uint8"):
        ssd.ssd_gated_scan(x, x, x, lam, reset=torch.zeros((1, 8), dtype=torch.bool))
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_gated_scan_backward(x, x, x, lam, torch.zeros((1, 2, 4)), x)
    ck = ssd.GatedCheckpoint8(1, 8, 4, device="cpu")
    with pytest.raises(ValueError, match="not both"):
        ssd.ssd_gated_scan(x, x, x, lam, states=st, checkpoint=ck)
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_gated_scan(x, x, x, lam, checkpoint=ssd.GatedCheckpoint8(1, 9, 4, device="cpu"))


def test_checkpoint_values():
    torch = pytest.importorskip("torch")
    import selective_state_space_12_b200 as ssd

    ck = ssd.GatedCheckpoint8(1, 66, 2, device="cpu")
    ck.q.fill_(3)
    ck.e.fill_(127)
    ck.e[0, 0, 1, 1] = 120          # 2^-7
    ck.e[1, 0, 0, 0] = 255
    x, r, i = ck.values()
    assert (x[0, :64] == 3).all() and (x[0, 64:, 1] == 3 / 128).all() and (x[0, 64:, 0] == 3).all()
    assert torch.isnan(r[0, :64, 0]).all() and (r[0, 64:] == 3).all() and (i == 3).all()
    assert ssd.gated_blocks(0) == 0 and ssd.gated_blocks(64) == 1 and ssd.gated_blocks(65) == 2
