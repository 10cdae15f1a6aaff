"""Which of their tensors the elementwise recurrences' calls may share: the end
state may take the initial one's place, nothing else (no GPU needed: refused
before anything is enqueued)."""
import itertools

import pytest

import test_gated_args as gated
import test_scan_backward_args as scan
from test_gated_args import INVALID, PTR, lib  # noqa: F401 (a fixture)


def refused(lib, status):
    said = lib.ssd_last_error().decode()
    assert status == INVALID and "aliases" in said, (status, said)


FWD = dict(h0=PTR["h0"], reset=PTR["reset"], hf=PTR["hf"], states=PTR["states"], q=PTR["q"],
           e=PTR["e"])
BWD = dict(reset=PTR["reset"], dhf=PTR["dhf"], dh0=PTR["dh0"])
SCAN = {n: 0x10000 * (k + 1) for k, n in enumerate(scan.NAMES)}


def test_forward(lib):
    outs, ins = ("y", "states", "q", "e", "hf"), ("x", "r", "i", "lam", "h0", "reset")
    for o, i in itertools.product(outs, ins):
        if (o, i) != ("hf", "h0"):
            refused(lib, gated.fwd(lib, **{**FWD, o: PTR[i]}))
    for o, p in itertools.combinations(outs, 2):
        refused(lib, gated.fwd(lib, **{**FWD, o: PTR[p]}))


def test_backward(lib):
    outs = ("dx", "dr", "di", "dlam", "dh0")
    for o, i in itertools.product(outs, ("x", "r", "i", "lam", "states", "dy", "dhf", "reset")):
        if (o, i) != ("dh0", "dhf"):
            refused(lib, gated.bwd(lib, **{**BWD, o: PTR[i]}))
    for o, i in itertools.product(outs, ("q", "e")):
        copies = dict(x=None, r=None, i=None, q=PTR["q"], e=PTR["e"])
        refused(lib, gated.bwd(lib, **{**BWD, **copies, o: PTR[i]}))
    for o, p in itertools.combinations(outs, 2):
        refused(lib, gated.bwd(lib, **{**BWD, o: PTR[p]}))


def test_step(lib):
    for o, i in (("y", "x"), ("y", "lam"), ("y", "h"), ("h", "x"), ("h", "r"), ("h", "lam")):
        refused(lib, gated.step(lib, **{o: PTR[i]}))


def test_scan_backward(lib):
    outs = ("dx", "ddt", "dA", "dB", "dC", "dD", "dbias", "dh0")
    ins = ("x", "dt", "A", "B", "C", "Dskip", "h0", "dy", "dhf")
    for o, i in itertools.product(outs, ins):
        if (o, i) != ("dh0", "dhf"):
            refused(lib, scan.call(lib, **{o: SCAN[i]}))
    for o, p in itertools.combinations(outs, 2):
        refused(lib, scan.call(lib, **{o: SCAN[p]}))


@pytest.mark.parametrize("call,kw", [
    (gated.fwd, {**FWD, "hf": PTR["h0"]}), (gated.bwd, {**BWD, "dh0": PTR["dhf"]}),
    (scan.call, {"dh0": SCAN["dhf"]})])
def test_the_end_in_the_starts_place_is_not_refused(lib, call, kw):
    """The next check, of the workspace, is the one that speaks."""
    assert call(lib, ws_bytes=1, **kw) == INVALID
    assert b"workspace" in lib.ssd_last_error()
