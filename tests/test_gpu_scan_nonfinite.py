"""The training scan with a NaN or an infinity in one element of an input: what the rule computes from it is not finite
(nothing hides it), and other sequences, other heads and what lies before it are what they were, bit for bit."""
import pytest
import torch

from helpers import DEV, say
from scan_reference import reference
from test_gpu_scan import backward, forward, inputs

pytestmark = pytest.mark.gpu
LENS, HQ, HV, B, T = [70, 200, 1, 33], 2, 4, 1, 100  # the element is in sequence B, at its token T
AT = sum(LENS[:B]) + T
CHUNK = slice(sum(LENS[:B]) + T // 64 * 64, min(sum(LENS[:B]) + T // 64 * 64 + 64, sum(LENS[:B + 1])))


def run(x, dout, dfinal, state):
    out, fin, tape = forward(x, LENS, state=True if state else None)
    return dict(backward(x, LENS, tape, dout, dfinal), out=out, final=fin)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "alpha", "beta", "dout", "dfinal", "state"])
def test_one_element(where, value, dtype):
    if where == "alpha" and value < 0:
        pytest.skip("gates are at least 0")
    say("non-finite", where, value, dtype)
    x, dout, dfinal = inputs(81, LENS, HQ, HV, 64, 48, dtype)
    clean = run(x, dout, dfinal, True)
    x, dout, dfinal = {n: t.clone() for n, t in x.items()}, dout.clone(), dfinal.clone()
    target = {"dout": dout, "dfinal": dfinal}.get(where, x.get(where))
    if where in ("state", "dfinal"):
        target[B, 1, 5, 7] = value
    elif where in ("alpha", "beta"):
        target[AT, 1] = value
    else:
        target[AT, 0 if where in ("q", "k") else 1, 5] = value
    got = run(x, dout, dfinal, True)
    want = reference(x, LENS, 1.0, dout, dfinal)
    # where the rule's results are not finite, these are not
    for n in got:
        lost = ~torch.isfinite(want[n]) & torch.isfinite(got[n]).cpu()
        assert not bool(lost.any()), (n, int(lost.sum()))
    # what may see it: value heads 0 and 1 (of q/k head 0), or head 1 alone
    heads = [0, 1] if where in ("q", "k") else [1]
    first, last = sum(LENS[:B]), sum(LENS[:B + 1])
    seen = {n: torch.zeros(t.shape, dtype=torch.bool, device=DEV) for n, t in got.items()}
    for h in heads:
        if where not in ("dout", "dfinal"):
            seen["out"][first if where == "state" else CHUNK.start:last, h] = True
            seen["final"][B, h] = True
        end = CHUNK.stop if where == "dout" else last
        for n in ("dv", "dalpha", "dbeta"):
            seen[n][first:end, h] = True
        for n in ("dq", "dk"):
            seen[n][first:end, h // 2] = True
        seen["dstate"][B, h] = True
    for n in got:
        assert torch.equal(got[n][~seen[n]], clean[n][~seen[n]]), n
