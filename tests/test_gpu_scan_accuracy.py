"""The training scan against float64 at the accuracy of its products: scan_model.BAR, which every lost partial product
would exceed (test_scan_model.py), and for results of fewer bits the exact result rounded to their type."""
import pytest
import torch

import scan_model as sm
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV, say
from scan_reference import reference
from test_gpu_scan import backward, forward, inputs

pytestmark = pytest.mark.gpu


def off(got, want):
    """Relative 2-norm of the difference from the exact result rounded to the type."""
    assert bool(torch.isfinite(got).all())
    want = want.to(got.dtype).double() if got.dtype != torch.float32 else want.double()
    return float((got.double().cpu() - want).norm() / want.norm())


def check(got, want, factor=1.0):
    worst = {n: off(got[n], want[n]) for n in got}
    say({n: f"{e:.1e}" for n, e in worst.items()})
    for n, e in worst.items():
        assert e <= factor * sm.typed_bar(got[n].dtype), (n, e)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d_k,d_v", [(64, 32), (128, 48), (32, 64)])
def test_every_product_has_its_parts(dtype, d_k, d_v):
    say("parts", dtype, d_k, d_v)
    x, dout, dfinal = sm.case(dtype, d_k=d_k, d_v=d_v)
    want = sm.exact(x, dout, dfinal)
    y = {n: (t[None, None] if n == "state" else t[:, None]).to(DEV).contiguous() for n, t in x.items()}
    for n in ("q", "k", "v"):
        y[n] = y[n].to(dtype)
    lens = [x["q"].shape[0]]
    out, fin, tape = forward(y, lens, torch.float32, sm.SCALE)
    got = backward(y, lens, tape, dout[:, None].to(DEV).contiguous(), dfinal[None, None].to(DEV).contiguous(), sm.SCALE)
    got.update(out=out, final=fin)
    check({n: t[0, 0] if n in ("final", "dstate") else t[:, 0] for n, t in got.items()}, want)


def whole(x, lens, scale, out_dtype, dout, dfinal):
    do = dout.to(out_dtype)
    out, fin, tape = forward(x, lens, out_dtype, scale)
    got = backward(x, lens, tape, do, dfinal, scale)
    got.update(out=out, final=fin)
    return got, reference(x, lens, scale, do, dfinal)


@pytest.mark.parametrize("lens,hq,hv,dk,dv", [
    ([63, 64, 65], 2, 4, 64, 32),
    ([130, 1, 0, 61], 3, 3, 64, 48),
    ([200], 1, 3, 128, 128),
    ([129, 5], 2, 4, 128, 80),
    ([170], 1, 5, 32, 256),
])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                             (torch.bfloat16, torch.float32), (torch.float32, torch.float16)])
def test_packed_sequences(lens, hq, hv, dk, dv, dtype, out_dtype):
    say("accuracy", lens, hq, hv, dk, dv, dtype, out_dtype)
    x, dout, dfinal = inputs(61, lens, hq, hv, dk, dv, dtype)
    check(*whole(x, lens, dk ** -0.5, out_dtype, dout, dfinal))


def test_two_value_tiles_a_workgroup():
    lens = [5, 64, 130, 33] * 10
    x, dout, dfinal = inputs(62, lens, 1, 3, 64, 80)
    assert len(lens) * 3 * 5 > 2 * 256
    check(*whole(x, lens, 0.125, torch.float32, dout, dfinal))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_segments(dtype):
    """Walks cut into segments: a state passes one more product, and so does its gradient."""
    lens = [1700]
    x, dout, dfinal = inputs(63, lens, 1, 2, 64, 32, dtype)
    check(*whole(x, lens, 0.125, torch.float32, dout, dfinal), factor=8 / 6)


@pytest.mark.parametrize("d_k", [32, 64, 128])
def test_products_lose_no_bits_to_one_side(d_k):
    """One token that only reads its state (alpha 1, beta 0): out = S q.  The values' parts multiply to the most that parts
    cut by truncation would lose, 3.9 2^-23 of the product.  Of the sum's roundings one per 32 indices is at its size, half
    a step each; the others and what the parts leave out are within another step."""
    c = 1 + 2.0 ** -7 - 2.0 ** -23
    x, _, _ = inputs(64, [1], 1, 2, d_k, 32)
    x["state"].fill_(c)
    x["q"].fill_(c)
    x["alpha"].fill_(1.0)
    x["beta"].fill_(0.0)
    out, _, _ = forward(x, [1])
    want = d_k * c * c  # exact in float64: 48 bits
    assert float(((out.double() - want) / want).abs().max()) <= (d_k // 32 + 2) * 2.0 ** -24


@pytest.mark.parametrize("power", [-104, 100])
def test_small_and_large_magnitudes(power):
    """The results are linear in v and the state, the gradients in dout and dfinal: every part of them stays in range."""
    lens = [130, 20]
    x, dout, dfinal = inputs(65, lens, 1, 2, 64, 32)
    x["v"] *= 2.0 ** power
    x["state"] *= 2.0 ** power
    check(*whole(x, lens, 0.125, torch.float32, dout * 2.0 ** min(0, -power), dfinal * 2.0 ** min(0, -power)))
    x, _, _ = inputs(65, lens, 1, 2, 64, 32)
    if power < 0:
        check(*whole(x, lens, 0.125, torch.float32, dout * 2.0 ** power, dfinal * 2.0 ** power))


def test_the_ends_of_the_range():
    x, _, _ = inputs(66, [1], 1, 2, 64, 32)
    x["alpha"].fill_(1.0)
    x["beta"].fill_(0.0)
    # what of a state lies below 2^-126 is lost: an output is off by that of each element, and by the sum's roundings
    x["state"] = torch.randn_like(x["state"]) * 2.0 ** -120
    out, fin, _ = forward(x, [1])
    want = (x["state"][0].double() @ x["q"][0, 0].double())
    lost = float(x["q"].abs().sum()) * 2.0 ** -126
    assert float((out[0].double() - want).abs().max()) <= lost + 2.0 ** -22 * float(x["state"].abs().max()) * 8
    assert torch.equal(fin, x["state"])
    # the largest values
    x["state"].fill_(3.38e38)
    x["q"].zero_()
    x["q"][0, 0, 5] = 0.5
    out, fin, _ = forward(x, [1])
    assert torch.equal(out, torch.full_like(out, 0.5 * 3.38e38)) and torch.equal(fin, x["state"])
