"""The training scan with gates of 0 and of next to nothing: what is forgotten leaves nothing behind, however large it
was, and such gates have their gradients."""
import pytest
import torch

import scan_model as sm
from gated_deltanet_recurrence_gdn_amd import binding as gb  # noqa: F401
from helpers import DEV, say
from scan_reference import reference
from test_gpu_scan import backward, forward, inputs

pytestmark = pytest.mark.gpu
HEADS = 4


def case(seed, T, at, value, d_k=64, d_v=32, dtype=torch.float32, size=1e25):
    """One sequence whose head h has the gate `value` at token at[h], and a state of `size` before it."""
    x, dout, dfinal = inputs(seed, [T], 2, HEADS, d_k, d_v, dtype)
    for h, t in enumerate(at):
        x["alpha"][t, h] = value
    x["state"] = torch.randn_like(x["state"]) * size
    return x, dout, dfinal


@pytest.mark.parametrize("d_k,d_v,dtype", [(64, 32, torch.float32), (128, 48, torch.bfloat16), (32, 16, torch.float32)])
@pytest.mark.parametrize("T,at", [(60, (0, 1, 30, 59)), (200, (0, 63, 64, 150)), (1700, (5, 127, 1000, 1699))])
def test_nothing_is_left_of_a_state(T, at, d_k, d_v, dtype):
    say("reset", T, at, d_k, d_v, dtype)
    x, dout, dfinal = case(71, T, at, 0.0, d_k, d_v, dtype)
    got, none = [], dict(x, state=torch.zeros_like(x["state"]))
    for y in (x, none):
        out, fin, tape = forward(y, [T])
        got.append(dict(backward(y, [T], tape, dout, dfinal), out=out, final=fin))
    a, b = got
    assert torch.equal(a["final"], b["final"])
    for h, t in enumerate(at):
        assert t > 0 or not bool(a["dstate"][0, h].any())  # forgotten before any token read it
        assert torch.equal(a["out"][t:, h], b["out"][t:, h]), h
        for n in ("dv", "dbeta"):
            assert torch.equal(a[n][t:, h], b[n][t:, h]), (n, h)
        assert torch.equal(a["dalpha"][t + 1:, h], b["dalpha"][t + 1:, h]), h
        if h % 2:  # the later one of a q/k head's two value heads
            for n in ("dq", "dk"):
                assert torch.equal(a[n][t:, h // 2], b[n][t:, h // 2]), (n, h)


def near(got, want, bar, what):
    e = float((got.double().cpu() - want).norm() / want.norm())
    assert e <= bar, (what, e)


@pytest.mark.parametrize("value", [0.0, 1e-30, 1e-42, 2.0 ** -61])
def test_small_gates_against_the_rule(value):
    """Before and after the gate each at its own scale: states of 1e10 before it, of order 1 after it."""
    T, at = 150, (10, 63, 64, 120)
    say("small gate", value)
    x, dout, dfinal = case(72, T, at, value, size=1e10)
    want = reference(x, [T], 0.5, dout, dfinal)
    out, fin, tape = forward(x, [T], scale=0.5)
    got = dict(backward(x, [T], tape, dout, dfinal, 0.5), out=out, final=fin)
    bar = 2 * sm.BAR  # of parts of the results, with decays of up to 2^-60
    for h, t in enumerate(at):
        for n in ("out", "dv", "dbeta"):
            near(got[n][t:, h], want[n][t:, h], bar, (n, h, "after"))
            near(got[n][:t, h], want[n][:t, h], bar, (n, h, "before"))
        near(got["dalpha"][t + 1:, h], want["dalpha"][t + 1:, h], bar, ("dalpha", h, "after"))
        near(got["dalpha"][:t, h], want["dalpha"][:t, h], bar, ("dalpha", h, "before"))
        g, w = float(got["dalpha"][t, h]), float(want["dalpha"][t, h])
        scale = float(want["dalpha"][:t, h].norm()) + abs(w)
        assert abs(g - w) <= bar * scale, (h, g, w)
        near(got["final"][0, h], want["final"][0, h], bar, ("final", h))
        near(got["dstate"][0, h], want["dstate"][0, h], bar, ("dstate", h))
    for n in ("dq", "dk"):
        for hq in range(2):
            t = max(at[2 * hq:2 * hq + 2])
            near(got[n][t:, hq], want[n][t:, hq], bar, (n, hq, "after"))


@pytest.mark.parametrize("share", [0.1, 0.5, 1.0])
def test_many_gates_of_zero(share):
    """Spans with none, one and several of them."""
    T = 200
    x, dout, dfinal = inputs(73, [T], 1, 3, 64, 48)
    g = torch.Generator(device=DEV).manual_seed(5)
    where = torch.rand(T, 3, generator=g, device=DEV) < share
    x["alpha"][where] = 0.0
    want = reference(x, [T], 0.5, dout, dfinal)
    out, fin, tape = forward(x, [T], scale=0.5)
    got = dict(backward(x, [T], tape, dout, dfinal, 0.5), out=out, final=fin)
    for n in got:
        if float(want[n].norm()) == 0:
            assert not bool(got[n].any()), n
        else:
            near(got[n], want[n], 2 * sm.BAR, n)
    for sel, what in ((where.cpu(), "zeros"), (~where.cpu(), "others")):
        if bool(sel.any()):
            near(got["dalpha"].cpu()[sel], want["dalpha"][sel], 2 * sm.BAR, what)
