"""What ssd_selective_scan_backward refuses, before anything is enqueued (no
GPU needed)."""
import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2
NAMES = ("x", "dt", "A", "B", "C", "Dskip", "h0", "dy", "dhf", "dx", "ddt", "dA", "dB", "dC", "dD",
         "dbias", "dh0")


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_12_b200 import build

    build.build()
    from selective_state_space_12_b200 import _lib

    return _lib.load()


def dims(**kw):
    from selective_state_space_12_b200 import _lib

    d = dict(batch=2, seqlen=100, nheads=64, headdim=1, dstate=16, ngroups=2, dtype=1, reserved=0)
    d.update(kw)
    return _lib.Dims(**d)


def call(lib, d=None, opts=None, ws=0x1000000, ws_bytes=1 << 40, **kw):
    a = {n: 0x10000 * (k + 1) for k, n in enumerate(NAMES)}
    a.update(kw)
    return lib.ssd_selective_scan_backward(*[a[n] for n in NAMES], ctypes.byref(d or dims()),
                                           opts, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(seqlen=-1), INVALID), (dict(headdim=16), INVALID),
    (dict(nheads=65), INVALID), (dict(dtype=3), INVALID), (dict(reserved=1), INVALID),
    (dict(dstate=12), UNSUPPORTED), (dict(dstate=32), UNSUPPORTED),
    (dict(batch=70000), UNSUPPORTED), (dict(nheads=(1 << 24) + 2), UNSUPPORTED),
    (dict(batch=60000, seqlen=1 << 30), UNSUPPORTED),
])
def test_sizes(lib, kw, status):
    assert call(lib, dims(**kw)) == status and lib.ssd_last_error()
    assert lib.ssd_selective_scan_backward_workspace_size(ctypes.byref(dims(**kw))) == 0


def test_pointers(lib):
    for n in NAMES:
        assert call(lib, **{n: 0x10001}) == INVALID, n
        if n not in ("Dskip", "h0", "dhf", "dD", "dbias", "dh0"):
            assert call(lib, **{n: None}) == INVALID, n
    for out in ("dx", "ddt", "dA", "dB", "dC", "dD", "dbias"):
        assert call(lib, **{out: 0x10000}) == INVALID and b"aliases" in lib.ssd_last_error()
    assert call(lib, dh0=0x10000 * 7) == INVALID  # h0 itself


def test_options_and_workspace(lib):
    from selective_state_space_12_b200 import _lib

    o = _lib.Options()
    o.discretization = 5
    assert call(lib, opts=ctypes.byref(o)) == INVALID
    o = _lib.Options()
    o.dt_min, o.dt_max = 2.0, 1.0
    assert call(lib, opts=ctypes.byref(o)) == INVALID
    need = lib.ssd_selective_scan_backward_workspace_size(ctypes.byref(dims()))
    assert need > 0
    assert call(lib, ws_bytes=need - 1) == INVALID
    assert call(lib, ws=0x1000010) == INVALID


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import selective_state_space_12_b200 as ssd

    x, A = torch.zeros((1, 8, 4)), -torch.ones((4, 16))
    B = torch.zeros((1, 8, 1, 16))
    f = ssd.ssd_selective_scan_backward
    with pytest.raises((ValueError, RuntimeError), match="(?i)cuda"):
        f(x, x, A, B, B, None, None, x)
    with pytest.raises(ValueError, match="shape"):
        f(x, x, A, B, B[:, :4].contiguous(), None, None, x)
    with pytest.raises(TypeError, match="dtype"):
        f(x, x, A, B, B, None, None, x.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        f(x, x, A, B, B, None, None, torch.zeros((1, 4, 8)).transpose(1, 2))
